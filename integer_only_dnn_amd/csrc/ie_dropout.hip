// Dropout of a (C, e) matrix, with an optional residual sum, from a
// counter-based generator: nothing is stored between the forward and the
// backward pass, both of which are this call with the same seed and step.
//
// Element (i, j) takes 16 bits of Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with key = seed
// and counter = (j / 8, i, step): one block of 128 bits serves eight
// neighbours of a row, the low half of a word first.  It is kept when the
// bits are at least `drop`, so with probability (65536 - drop) / 65536, and
// then scaled by s = 65536 / (65536 - drop), held to 24 bits:
//   y = C s 2^e [kept] + R,
// the sum held to 53 bits (exact while the terms span no more), rounded once
// into Y's groups.
//
// Bound by its instructions, 23 an element with a residual (the generator's among
// them: 10 rounds of two 32 x 32 -> 64 bit products for eight elements; 72 % of
// the cycles issue one), beside the stream over X, R and Y: 25216 x 768 with a residual takes 18 us,
// 11 of them its 58 MB at the rate of a large copy.
#include "ie_f64.h"
#include "ie_internal.h"

#pragma clang fp contract(off)

namespace ie {

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

struct Philox {
    uint32_t k0[10], k1[10];
    uint32_t c2, c3;
    __device__ __forceinline__ void init(const DropArgs &p) {
        const uint64_t step = p.step + (p.step_ptr ? *p.step_ptr : 0);
        c2 = (uint32_t)step;
        c3 = (uint32_t)(step >> 32);
        k0[0] = (uint32_t)p.seed;
        k1[0] = (uint32_t)(p.seed >> 32);
#pragma unroll
        for (int i = 1; i < 10; ++i) {
            k0[i] = k0[i - 1] + 0x9E3779B9u;
            k1[i] = k1[i - 1] + 0xBB67AE85u;
        }
    }
    // Which of the eight elements of block `b` of row `row` are kept, as bytes
    // of all ones or zeros.
    __device__ __forceinline__ void keep(uint32_t b, uint32_t row, uint32_t drop, uint32_t (&m)[2]) const {
        uint32_t a0 = b, a1 = row, a2 = c2, a3 = c3;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = (uint64_t)a0 * 0xD2511F53u, p1 = (uint64_t)a2 * 0xCD9E8D57u;
            a0 = __builtin_amdgcn_bitop3_b32((uint32_t)(p1 >> 32), a1, k0[i], 0x96);  // xor of three
            a2 = __builtin_amdgcn_bitop3_b32((uint32_t)(p0 >> 32), a3, k1[i], 0x96);
            a1 = (uint32_t)p1;
            a3 = (uint32_t)p0;
        }
        m[0] = __builtin_amdgcn_perm(keep2(a1, drop), keep2(a0, drop), 0x06040200u);
        m[1] = __builtin_amdgcn_perm(keep2(a3, drop), keep2(a2, drop), 0x06040200u);
    }
    // Halves of all ones where those of u are at least drop (drop - u, clamped
    // at 0, is 0 there).
    static __device__ __forceinline__ uint32_t keep2(uint32_t u, uint32_t drop) {
        const us2 one = {1, 1}, d = {(unsigned short)drop, (unsigned short)drop};
        const us2 z = __builtin_elementwise_min(__builtin_elementwise_sub_sat(d, __builtin_bit_cast(us2, u)), one) - one;
        return __builtin_bit_cast(uint32_t, z);
    }
};

// The values of four kept mantissas w and residual mantissas r.  Both products
// are exact, so this is one rounded sum.
template <bool RES>
__device__ __forceinline__ void drop4(uint32_t w, uint32_t r, double sx, double sr, double *y) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        y[k] = RES ? __builtin_fma((double)byte_of(w, k), sx, (double)byte_of(r, k) * sr) : (double)byte_of(w, k) * sx;
}

__device__ __forceinline__ uint32_t round4(const double *y, double inv) {
    return pack4(mant_of(y[0], inv), mant_of(y[1], inv), mant_of(y[2], inv), mant_of(y[3], inv));
}

// The exponent of a whole-tensor result from the blocks' needs.
template <int BT>
__device__ __forceinline__ double whole_inv(const DropArgs &p, int *sh) {
    int m = NEED_NONE;
    for (int i = threadIdx.x; i < p.n_bmax; i += BT) m = max(m, p.bmax[i]);
    m = row_reduce<BT>(m, Max{}, sh);
    const int e = clamp_exp_flag(max(E_MIN, m), p.flags);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.ye[0] = (int8_t)e;
    return pow2(-e);
}

// T threads per row, E elements (a multiple of 8) per thread; the next row's
// loads are in flight while a row is computed.  A whole-tensor result takes
// two launches: the first leaves the kept mantissas in Y, so that the second
// draws nothing.
template <int T, int E, bool RES>
__global__ __launch_bounds__(T > 256 ? T : 256) void dropout_kernel(DropArgs p) {
    using C = Cols<T, E>;
    constexpr int BT = T > 256 ? T : 256, RPB = BT / T, W = E / 4;
    __shared__ int shi[BT / 64];
    const int t = threadIdx.x % T, slot = threadIdx.x / T, n = p.cols;
    const long long step = (long long)gridDim.x * RPB;
    const int8_t *src = p.mode == NORM_ROUND ? p.y : p.x;
    C cols;
    cols.init(t, n);
    uint32_t w[W], w_next[W], r[RES ? W : 1], r_next[RES ? W : 1];
    int ex = 0, er = 0, ex_next = 0, er_next = 0;
    // threads past the end repeat the last row
    auto fetch = [&](long long r0) {
        const long long row = min(r0 + slot, p.rows - 1);
        const bool whole = n % C::CH == 0 || r0 + RPB + C::CH <= p.rows;
        cols.load(src + row * n, whole, w_next);
        ex_next = p.xe[p.x_row ? row : 0];
        if constexpr (RES) {
            cols.load(p.r + row * n, whole, r_next);
            er_next = p.re[p.r_row ? row : 0];
        }
    };
    fetch((long long)blockIdx.x * RPB);
    Philox g;
    g.init(p);
    double inv = p.mode == NORM_ROUND ? whole_inv<BT>(p, shi) : 0.0;
    int run = 0;  // high word of the largest magnitude (NORM_NEED)
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += step) {
        const long long row = min(r0 + slot, p.rows - 1);
        const bool ok = r0 + slot < p.rows;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = w_next[i];
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < W; ++i) r[i] = r_next[i];
        }
        ex = ex_next;
        er = er_next;
        if (r0 + step < p.rows) fetch(r0 + step);
        if (p.mode != NORM_ROUND) {
#pragma unroll
            for (int i = 0; i < W; i += 2) {
                uint32_t m[2];
                g.keep((uint32_t)cols.col(4 * i) >> 3, (uint32_t)row, p.drop, m);
                w[i] &= m[0];
                w[i + 1] &= m[1];
            }
        }
        cols.clear(w);
        if constexpr (RES) cols.clear(r);
        if (p.mode == NORM_NEED && ok) cols.store(p.y + row * n, w);
        const double sx = p.scale * pow2(ex), sr = pow2(er);
        double y[E];
        MaxMag mx;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            drop4<RES>(w[i], RES ? r[i] : 0u, sx, sr, y + 4 * i);
            mx.add(y[4 * i], y[4 * i + 1]);
            mx.add(y[4 * i + 2], y[4 * i + 3]);
        }
        if (p.mode == NORM_NEED) {
            run = max(run, mx.word());
            continue;
        }
        if (p.mode == NORM_ROWS) {
            int e = max(E_MIN, need_word(row_reduce<T>(mx.word(), Max{}, shi), p.q));
            if (ok && t == 0) {
                e = clamp_exp_flag(e, p.flags);
                p.ye[row] = (int8_t)e;
            }
            inv = pow2(-min(e, E_MAX));
        }
        if (!ok) continue;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = round4(y + 4 * i, inv);
        cols.store(p.y + row * n, w);
    }
    if (p.mode == NORM_NEED) {
        run = row_reduce<BT>(run, Max{}, shi);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = need_word(run, p.q);
    }
}

// Rows too long to be held (2000 x 24576 with a residual 62 us, 500 x 100000 58,
// where their bytes take 29 at the rate of a large copy; one row of 2^24 3.4 ms,
// for it has one block): one block per row walks it twice, for its largest
// value (leaving the kept mantissas in Y) and to round it (a whole-tensor
// result: once per launch).
template <bool RES>
__global__ __launch_bounds__(1024) void dropout_long_kernel(DropArgs p) {
    __shared__ int shi[16];
    const int n = p.cols;
    Philox g;
    g.init(p);
    double inv = p.mode == NORM_ROUND ? whole_inv<1024>(p, shi) : 0.0;
    int run = 0;
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int8_t *x = p.x + row * n, *r = RES ? p.r + row * n : nullptr;
        int8_t *out = p.y + row * n;
        const double sx = p.scale * pow2((int)p.xe[p.x_row ? row : 0]);
        const double sr = RES ? pow2((int)p.re[p.r_row ? row : 0]) : 0.0;
        uint32_t w[2], rw[2] = {0, 0};
        double y[8];
        if (p.mode != NORM_ROUND) {
            MaxMag mx;
            for (long long c = 8ll * threadIdx.x; c < n; c += 8192) {
                uint32_t m[2];
                load_run<8>(x, (int)c, n, w);
                if constexpr (RES) load_run<8>(r, (int)c, n, rw);
                g.keep((uint32_t)c >> 3, (uint32_t)row, p.drop, m);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[i] &= m[i];
                    drop4<RES>(w[i], rw[i], sx, sr, y + 4 * i);
                }
                store_run<8>(out, (int)c, n, w);
#pragma unroll
                for (int k = 0; k < 8; k += 2) mx.add(y[k], y[k + 1]);
            }
            if (p.mode == NORM_NEED) {
                run = max(run, mx.word());
                continue;
            }
            int e = max(E_MIN, need_word(row_reduce<1024>(mx.word(), Max{}, shi), p.q));
            if (threadIdx.x == 0) {
                e = clamp_exp_flag(e, p.flags);
                p.ye[row] = (int8_t)e;
            }
            inv = pow2(-min(e, E_MAX));
        }
        for (long long c = 8ll * threadIdx.x; c < n; c += 8192) {
            load_run<8>(out, (int)c, n, w);
            if constexpr (RES) load_run<8>(r, (int)c, n, rw);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                drop4<RES>(w[i], rw[i], sx, sr, y + 4 * i);
                w[i] = round4(y + 4 * i, inv);
            }
            store_run<8>(out, (int)c, n, w);
        }
    }
    if (p.mode == NORM_NEED) {
        run = row_reduce<1024>(run, Max{}, shi);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = need_word(run, p.q);
    }
}

hipError_t launch_dropout(const DropArgs &a, const NormPlan &pl, hipStream_t st) {
    if (!dropout_built(pl)) return hipErrorInvalidValue;
    prof_begin(st, PROF_DROPOUT);
    if (pl.e == 0) {
        if (a.r) hipLaunchKernelGGL(dropout_long_kernel<true>, dim3(pl.grid), dim3(1024), 0, st, a);
        else hipLaunchKernelGGL(dropout_long_kernel<false>, dim3(pl.grid), dim3(1024), 0, st, a);
    }
#define IE_CASE(T_, E_)                                                                                 \
    if (pl.t == T_ && pl.e == E_) {                                                                     \
        const dim3 grid(pl.grid), block(T_ > 256 ? T_ : 256);                                           \
        if (a.r) hipLaunchKernelGGL((dropout_kernel<T_, E_, true>), grid, block, 0, st, a);             \
        else hipLaunchKernelGGL((dropout_kernel<T_, E_, false>), grid, block, 0, st, a);                \
    }
    IE_DROP_SHAPES(IE_CASE)
#undef IE_CASE
    prof_end(st, PROF_DROPOUT);
    return hipGetLastError();
}

}  // namespace ie
