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
// A stream over X, R and Y: 10 rounds of two 32 x 32 -> 64 bit products are
// 2.5 products an element, which run beside the loads and stores.
#include "ie_f64.h"
#include "ie_internal.h"

#pragma clang fp contract(off)

namespace ie {

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
    // The 128 bits of block `b` of row `row`.
    __device__ __forceinline__ void block(uint32_t b, uint32_t row, uint32_t (&u)[4]) const {
        uint32_t a0 = b, a1 = row, a2 = c2, a3 = c3;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p0 = (uint64_t)a0 * 0xD2511F53u, p1 = (uint64_t)a2 * 0xCD9E8D57u;
            a0 = (uint32_t)(p1 >> 32) ^ a1 ^ k0[i];
            a2 = (uint32_t)(p0 >> 32) ^ a3 ^ k1[i];
            a1 = (uint32_t)p1;
            a3 = (uint32_t)p0;
        }
        u[0] = a0;
        u[1] = a1;
        u[2] = a2;
        u[3] = a3;
    }
};

// The eight results from column c of a row (zeros past its end): sx, sr are
// the scaled exponents of X and R.
__device__ __forceinline__ void drop8(const DropArgs &p, const Philox &g, const int8_t *x, const int8_t *r, int c,
                                      uint32_t row, double sx, double sr, double (&y)[8]) {
    const int n = p.cols;
    uint32_t u[4];
    g.block((uint32_t)c >> 3, row, u);
    const uint32_t xw[2] = {load4(x, c, n), load4(x, c + 4, n)};
    uint32_t rw[2] = {0, 0};
    if (r) {
        rw[0] = load4(r, c, n);
        rw[1] = load4(r, c + 4, n);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t bits = k & 1 ? u[k >> 1] >> 16 : u[k >> 1] & 0xffffu;
        const int v = bits >= p.drop ? byte_of(xw[k >> 2], k & 3) : 0;
        // both products are exact, so this is one rounded sum
        y[k] = __builtin_fma((double)v, sx, (double)byte_of(rw[k >> 2], k & 3) * sr);
    }
}

__device__ __forceinline__ void put8(int8_t *row, int c, int n, const double (&y)[8], double inv) {
    store4(row, c, n, pack4(mant_of(y[0], inv), mant_of(y[1], inv), mant_of(y[2], inv), mant_of(y[3], inv)));
    store4(row, c + 4, n, pack4(mant_of(y[4], inv), mant_of(y[5], inv), mant_of(y[6], inv), mant_of(y[7], inv)));
}

// T threads per row, E elements (a multiple of 8) per thread.
template <int T, int E>
__global__ __launch_bounds__(T > 256 ? T : 256) void dropout_kernel(DropArgs p) {
    constexpr int BT = T > 256 ? T : 256, RPB = BT / T, W = E / 8;
    __shared__ int shi[BT / 64];
    const int t = threadIdx.x % T, slot = threadIdx.x / T, n = p.cols;
    Philox g;
    g.init(p);
    double inv = 0.0;
    if (p.mode == NORM_ROUND) {
        int m = NEED_NONE;
        for (int i = threadIdx.x; i < p.n_bmax; i += BT) m = max(m, p.bmax[i]);
        m = row_reduce<BT>(m, Max{}, shi);
        const int e = clamp_exp_flag(max(E_MIN, m), p.flags);
        inv = pow2(-e);
        if (blockIdx.x == 0 && threadIdx.x == 0) p.ye[0] = (int8_t)e;
    }
    int run = 0;  // high word of the largest magnitude (NORM_NEED)
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += (long long)gridDim.x * RPB) {
        const long long row = min(r0 + slot, p.rows - 1);  // threads past the end repeat the last row
        const bool ok = r0 + slot < p.rows;
        const int8_t *x = p.x + row * n, *r = p.r ? p.r + row * n : nullptr;
        const double sx = p.scale * pow2((int)p.xe[p.x_row ? row : 0]);
        const double sr = r ? pow2((int)p.re[p.r_row ? row : 0]) : 0.0;
        double y[W][8];
        MaxMag mx;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int c = 8 * (i * T + t);
            if (c < n) {
                drop8(p, g, x, r, c, (uint32_t)row, sx, sr, y[i]);
#pragma unroll
                for (int k = 0; k < 8; k += 2) mx.add(y[i][k], y[i][k + 1]);
            }
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
        for (int i = 0; i < W; ++i) {
            const int c = 8 * (i * T + t);
            if (c < n) put8(p.y + row * n, c, n, y[i], inv);
        }
    }
    if (p.mode == NORM_NEED) {
        run = row_reduce<BT>(run, Max{}, shi);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = need_word(run, p.q);
    }
}

// Rows too long to be held: one block per row walks it twice, for its largest
// value and to round it (a whole-tensor result: once per launch).
__global__ __launch_bounds__(1024) void dropout_long_kernel(DropArgs p) {
    __shared__ int shi[16];
    const int n = p.cols;
    Philox g;
    g.init(p);
    double inv = 0.0;
    int run = 0;
    if (p.mode == NORM_ROUND) {
        int m = NEED_NONE;
        for (int i = threadIdx.x; i < p.n_bmax; i += 1024) m = max(m, p.bmax[i]);
        m = row_reduce<1024>(m, Max{}, shi);
        const int e = clamp_exp_flag(max(E_MIN, m), p.flags);
        inv = pow2(-e);
        if (blockIdx.x == 0 && threadIdx.x == 0) p.ye[0] = (int8_t)e;
    }
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int8_t *x = p.x + row * n, *r = p.r ? p.r + row * n : nullptr;
        const double sx = p.scale * pow2((int)p.xe[p.x_row ? row : 0]);
        const double sr = r ? pow2((int)p.re[p.r_row ? row : 0]) : 0.0;
        double y[8];
        if (p.mode != NORM_ROUND) {
            MaxMag mx;
            for (long long c = 8ll * threadIdx.x; c < n; c += 8192) {
                drop8(p, g, x, r, (int)c, (uint32_t)row, sx, sr, y);
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
            drop8(p, g, x, r, (int)c, (uint32_t)row, sx, sr, y);
            put8(p.y + row * n, (int)c, n, y, inv);
        }
    }
    if (p.mode == NORM_NEED) {
        run = row_reduce<1024>(run, Max{}, shi);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = need_word(run, p.q);
    }
}

#define IE_DROP_SHAPES(X) \
    X(8, 8) X(8, 16) X(8, 24) X(16, 16) X(16, 24) X(32, 16) X(32, 24) X(64, 16) X(64, 24) X(256, 8) X(256, 16) \
    X(256, 24) X(1024, 8) X(1024, 16) X(1024, 24)

hipError_t launch_dropout(const DropArgs &a, const NormPlan &pl, hipStream_t st) {
    prof_begin(st, PROF_DROPOUT);
    if (pl.e == 0) hipLaunchKernelGGL(dropout_long_kernel, dim3(pl.grid), dim3(1024), 0, st, a);
#define IE_CASE(T_, E_)                                                                                         \
    if (pl.t == T_ && pl.e == E_)                                                                               \
        hipLaunchKernelGGL((dropout_kernel<T_, E_>), dim3(pl.grid), dim3(T_ > 256 ? T_ : 256), 0, st, a);
    IE_DROP_SHAPES(IE_CASE)
#undef IE_CASE
    prof_end(st, PROF_DROPOUT);
    return hipGetLastError();
}

}  // namespace ie
