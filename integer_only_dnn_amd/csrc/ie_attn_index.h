// Which tile of which sequence, and which head, a workgroup of attention takes.
// Plain arithmetic over a wave's lanes, for the kernels and for a check on the
// host: `Lanes` evaluates a function in every lane (each, ballot), and reads, adds up and
// compares what that gave (of, at, sum, max).
#pragma once

#include <stdint.h>

#include "ie_plan.h"

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define IE_BOTH __host__ __device__ __forceinline__
#else
#define IE_BOTH inline
#endif

namespace ie {

IE_BOTH int lower(int a, int b) { return a < b ? a : b; }
IE_BOTH int upper(int a, int b) { return a > b ? a : b; }

// Sequence s of a packed batch: its rows [a, b).  Offsets are read on the
// device; bounds that lie outside the matrix or before the last one are
// clipped, a sequence longer than `most` is cut there.
struct Span {
    int a, n;
};
template <class P>
IE_BOTH Span span_of(const P &p, int x, int y) {
    const int rows = (int)p.rows;
    const int a = lower(upper(x, 0), rows), b = lower(upper(y, a), rows);
    return Span{a, lower(b - a, p.most)};
}

// Tiles of BM rows: sequence s owns the slots from off[s] / BM + s on, enough
// for its ceil(n / BM) tiles whatever the other lengths are, so that a slot
// finds its sequence by a search, 64 offsets a turn, and nothing is laid out
// beforehand.  Returns the sequence's rows and the tile's first row in it (>= n:
// no such tile).
template <class Lanes, class P>
IE_BOTH Span slot_span(const Lanes &w, const P &p, int slot, int bm, int &first) {
    if (!p.off) {
        first = slot * bm;
        return Span{0, lower((int)p.rows, p.most)};
    }
    int lo = 0, len = p.n_seq, step, k;
    typename Lanes::Int x, y;
    do {
        step = (len + 63) >> 6;
        auto seq = [&](int lane) { return lower(lo + lane * step, p.n_seq - 1); };
        x = w.each([&](int lane) { return p.off[seq(lane)]; });
        y = w.each([&](int lane) { return p.off[seq(lane) + 1]; });
        const uint64_t below = w.ballot([&](int lane) {
            return lane * step < len && upper(w.of(x, lane), 0) / bm + lo + lane * step <= slot;
        });
        k = below ? 63 - __builtin_clzll(below) : 0;
        lo += k * step;
        len = lower(step, len - k * step);
    } while (step > 1);
    const int from = w.at(x, k);
    const Span s = span_of(p, from, w.at(y, k));
    const int at = slot - (upper(from, 0) / bm + lo);
    first = at < 0 || at > s.n / bm ? s.n : at * bm;
    return s;
}

// A launch's items: the tiles of every key head, and of each the `per` query
// heads that share it.  Workgroups reach the XCDs in turn (blockIdx % 8).  In
// general an XCD takes every eighth pair (tile, key head), tiles in order, the
// heads of a pair one behind the other: they share its L2, and every XCD meets
// heavy and light tiles alike.  Short sequences: it takes `chunk` pairs in a row,
// then skips the others' seven chunks, so that the few tiles of a sequence read
// its keys from one L2 (128 x 197 tokens, 12 heads of 64: forward pass 70 -> 67
// us, dK and dV 135 -> 127).
struct Item {
    int rank, kvh, gh;
};
template <class P>
IE_BOTH Item att_item(const P &p, int per, int block, int grid) {
    const int idx = block >> 3, xcd = block & 7, v = idx / per;
    int u = 8 * v + xcd;
    if (p.chunk) {
        const int all = grid / 8 / per, turn = v / p.chunk, at = turn * p.chunk;
        u = 8 * at + xcd * lower(p.chunk, all - at) + v - at;
    }
    return Item{u / p.kv, u % p.kv, idx - v * per};
}
inline unsigned att_grid(long long tiles, int kv, int per) { return (unsigned)((tiles * kv + 7) / 8 * 8 * per); }
// Pairs of a chunk: equal parts of up to 16 tiles, where sequences have up to 16
// tiles on the average and all tiles of one are alike; else 0.
inline int att_chunk(long long rows, int n_seq, int kv, int bm, bool alike) {
    const long long slots = att_slots(rows, n_seq, bm), each = (slots * kv + 7) / 8;
    if (!alike || rows > 16ll * bm * n_seq) return 0;
    const long long turns = (each + 16 * kv - 1) / (16 * kv);
    return (int)((each + turns - 1) / turns);
}

// The tile of a rank: its sequence and its number in it; false: none.  Tiles of
// a causal launch differ in work (the t-th of a sequence meets t + 1 tiles of
// keys): the heaviest come first, for up to 64 sequences (a lane each); else
// sequences in order, each with enough ranks for its tiles (see slot_span).
template <bool HEAVY, class Lanes, class P>
IE_BOTH bool rank_tile(const Lanes &w, const P &p, int rank, int bm, Span &sp, int &tile) {
    if (!HEAVY || !p.off || p.n_seq > 64) {
        int first;
        const int slots = (int)(p.rows / bm) + upper(p.n_seq, 1);
        sp = slot_span(w, p, HEAVY ? slots - 1 - rank : rank, bm, first);
        tile = first / bm;
        return rank < slots && first < sp.n;
    }
    const auto a = w.each([&](int lane) { return lane < p.n_seq ? span_of(p, p.off[lane], p.off[lane + 1]).a : 0; });
    const auto n = w.each([&](int lane) { return lane < p.n_seq ? span_of(p, p.off[lane], p.off[lane + 1]).n : 0; });
    const auto tiles = w.each([&](int lane) { return (w.of(n, lane) + bm - 1) / bm; });
    // tiles whose number is t or more: A(t) = sum max(0, tiles - t)
    auto at_least = [&](int t) { return w.sum(w.each([&](int lane) { return upper(0, w.of(tiles, lane) - t); })); };
    int lo = 0, hi = w.max(tiles);  // A(lo) > rank >= A(hi)
    if (rank >= at_least(0)) return false;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at_least(mid) > rank) lo = mid;
        else hi = mid;
    }
    // the k-th sequence with a tile of number lo
    int k = rank - at_least(lo + 1);
    uint64_t have = w.ballot([&](int lane) { return w.of(tiles, lane) > lo; });
    while (k-- > 0) have &= have - 1;
    const int s = __builtin_ctzll(have);
    sp.a = w.at(a, s);
    sp.n = w.at(n, s);
    tile = lo;
    return true;
}

}  // namespace ie
