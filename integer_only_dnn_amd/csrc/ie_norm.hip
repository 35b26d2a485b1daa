// Layer norm of (C, e) rows, forward and backward, and the column sums of a
// gradient (the weight and bias gradients of the norm, the bias gradient of a
// linear layer).
//
// A row of N mantissas C at exponent e, S = sum C, V = N sum C^2 - S^2 (exact
// integers, V < 2^43):
//   T = V + N^2 eps 2^(-2e),  r = 1 / sqrt(T)  (0 when T = 0),
//   d = N C - S (exact),      h = d r = (x - mean) / sqrt(var + eps),
//   y = h gamma + beta, rounded once into Y's groups.
// Backward, with g = dY gamma' (gamma re-expressed at its largest exponent)
// and f = h at 2^-20, rounded half to even:
//   G1 = sum g, G2 = sum g f (exact),  z = (N g - G1) - f (G2 2^-40),
//   dX = z r 2^(e_dY + e_gamma' - e_X),
//   dgamma = sum_rows a f 2^(e* - 20),  dbeta = sum_rows a 2^e*,
// a = dY re-expressed at the largest of its row exponents e*.
//
// Integers are held in the fp64 unit, whose fused multiply-add runs at the
// fp32 rate on this chip: every integer above stays below 2^53 (|g f| sums to
// at most N 2^34 by Cauchy, since sum f^2 <= N 2^40), so those steps are
// exact in any order and the results do not depend on how rows are split
// over lanes, blocks or launches.  T, r, h, the products and sums of y and z
// and z r are single operations rounded to 53 bits, half to even; no
// contraction is allowed in this file, so each of them rounds by itself.
#include "ie_f64.h"
#include "ie_internal.h"

#pragma clang fp contract(off)

namespace ie {

struct RowStat {
    double s, r;  // sum of the mantissas, 1 / sqrt(T)
};

// The statistics of a row held four mantissas to a word (zeros past its end).
template <int T, int W>
__device__ __forceinline__ RowStat row_stat(const uint32_t (&w)[W], int n, double n2eps, int eps_e, int e, int *shi) {
    int s = 0, q = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        s = __builtin_amdgcn_sdot4((int)w[i], 0x01010101, s, false);
        q = __builtin_amdgcn_sdot4((int)w[i], (int)w[i], q, false);
    }
    s = row_reduce<T>(s, Add{}, shi);
    q = row_reduce<T>(q, Add{}, shi);
    const double sd = (double)s, v = (double)n * (double)q - sd * sd;  // exact: V < 2^43
    const double t = v + n2eps * pow2(eps_e - 2 * e);
    return RowStat{sd, t > 0.0 ? 1.0 / __builtin_sqrt(t) : 0.0};
}

// The value of channel c of a parameter vector.
__device__ __forceinline__ double channel(const NormVec &v, int c) {
    return (double)v.m[c] * pow2((int)v.e[v.per ? c : 0]);
}

// T threads per row, E elements per thread: thread t holds columns
// 4 (i T + t) + k, i < E / 4, k < 4.
template <int T, int E>
__global__ __launch_bounds__(T > 256 ? T : 256) void norm_fwd_kernel(NormFwd p) {
    constexpr int BT = T > 256 ? T : 256, RPB = BT / T, W = E / 4;
    __shared__ int shi[BT / 64];
    __shared__ double shd[BT / 64];
    const int t = threadIdx.x % T, slot = threadIdx.x / T, n = p.cols;
    double gam[E], bet[E];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = 4 * (i * T + t) + k;
            // past the row both are zero, so y is
            gam[4 * i + k] = c < n ? (p.gamma.m ? channel(p.gamma, c) : 1.0) : 0.0;
            bet[4 * i + k] = c < n && p.beta.m ? channel(p.beta, c) : 0.0;
        }
    double inv = 0.0;  // of a whole-tensor result
    if (p.mode == NORM_ROUND) {
        int m = NEED_NONE;
        for (int i = threadIdx.x; i < p.n_bmax; i += BT) m = max(m, p.bmax[i]);
        m = row_reduce<BT>(m, Max{}, shi);
        const int e = clamp_exp_flag(max(E_MIN, m), p.flags);
        inv = pow2(-e);
        if (blockIdx.x == 0 && threadIdx.x == 0) p.oe[0] = (int8_t)e;
    }
    double run = 0.0;  // largest magnitude of this thread's rows (NORM_NEED)
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += (long long)gridDim.x * RPB) {
        const long long row = r0 + slot;
        const bool ok = row < p.rows;
        const int8_t *x = p.x + (ok ? row : 0) * n;
        uint32_t w[W];
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = ok ? load4(x, 4 * (i * T + t), n) : 0u;
        const int e = p.xe[p.x_row && ok ? row : 0];
        const RowStat st = row_stat<T>(w, n, p.n2eps, p.eps_e, e, shi);
        double y[E], mx = 0.0;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const double d = __builtin_fma((double)byte_of(w[j / 4], j % 4), (double)n, -st.s);
            y[j] = (d * st.r) * gam[j] + bet[j];
            mx = fmax(mx, fabs(y[j]));
        }
        if (p.mode == NORM_NEED) {
            if (ok) run = fmax(run, mx);
            continue;
        }
        if (p.mode == NORM_ROWS) {
            mx = row_reduce<T>(mx, Max{}, shd);
            int ex = max(E_MIN, need_f64(mx, p.q));
            if (ok && t == 0) {
                ex = clamp_exp_flag(ex, p.flags);
                p.oe[row] = (int8_t)ex;
            }
            inv = pow2(-min(ex, E_MAX));
        }
        if (!ok) continue;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int c = 4 * (i * T + t);
            if (c < n)
                store4(p.out + row * n, c, n,
                       pack4(mant_of(y[4 * i], inv), mant_of(y[4 * i + 1], inv), mant_of(y[4 * i + 2], inv),
                             mant_of(y[4 * i + 3], inv)));
        }
    }
    if (p.mode == NORM_NEED) {
        run = row_reduce<BT>(run, Max{}, shd);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = need_f64(run, p.q);
    }
}

// Backward: the same layout.  NORM_NEED and NORM_ROWS also add up the columns
// of dgamma and dbeta (p.pf, p.pb: one row of partial sums per block).
template <int T, int E>
__global__ __launch_bounds__(T > 256 ? T : 256) void norm_bwd_kernel(NormBwd p) {
    constexpr int BT = T > 256 ? T : 256, RPB = BT / T, W = E / 4;
    __shared__ int shi[BT / 64];
    __shared__ double shd[BT / 64];
    const int t = threadIdx.x % T, slot = threadIdx.x / T, n = p.cols;
    const int gtop = p.gamma.m ? p.top[1] : 0;  // exponent of the re-expressed gamma
    const int dtop = p.top[0];                  // largest exponent of dY
    const bool sums = p.pf && p.mode != NORM_ROUND, grad = p.out != nullptr;
    double gam[E];
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = 4 * (i * T + t) + k;
            double v = c < n ? 1.0 : 0.0;
            if (p.gamma.m && c < n) v = (double)rne_shift32(p.gamma.m[c], gtop - (int)p.gamma.e[p.gamma.per ? c : 0]);
            gam[4 * i + k] = v;
        }
    double inv = 0.0;
    if (p.mode == NORM_ROUND) {
        int m = NEED_NONE;
        for (int i = threadIdx.x; i < p.n_bmax; i += BT) m = max(m, p.bmax[i]);
        m = row_reduce<BT>(m, Max{}, shi);
        const int e = clamp_exp_flag(max(E_MIN, m), p.flags);
        inv = pow2(-e);
        if (blockIdx.x == 0 && threadIdx.x == 0) p.oe[0] = (int8_t)e;
    }
    double af[E];
    int ab[E];
#pragma unroll
    for (int j = 0; j < E; ++j) af[j] = 0.0, ab[j] = 0;
    double run = 0.0;
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += (long long)gridDim.x * RPB) {
        const long long row = r0 + slot;
        const bool ok = row < p.rows;
        const long long off = (ok ? row : 0) * n;
        uint32_t w[W], v[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            w[i] = ok ? load4(p.x + off, 4 * (i * T + t), n) : 0u;
            v[i] = ok ? load4(p.dy + off, 4 * (i * T + t), n) : 0u;
        }
        const int ex = p.xe[p.x_row && ok ? row : 0], ey = p.dye[p.dy_row && ok ? row : 0];
        const RowStat st = row_stat<T>(w, n, p.n2eps, p.eps_e, ex, shi);
        const double r20 = st.r * 1048576.0;  // h 2^20 = d (r 2^20)
        double f[E], g[E], g1 = 0.0, g2 = 0.0;
        const int sh = dtop - ey;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const double d = __builtin_fma((double)byte_of(w[j / 4], j % 4), (double)n, -st.s);
            const int c = byte_of(v[j / 4], j % 4);
            f[j] = rint_magic(d * r20);
            g[j] = (double)c * gam[j];
            g1 += g[j];
            g2 = __builtin_fma(g[j], f[j], g2);
            if (sums) {
                const int a = rne_shift32(c, sh);
                af[j] = __builtin_fma((double)a, f[j], af[j]);
                ab[j] += a;
            }
        }
        if (!grad) continue;
        g1 = row_reduce<T>(g1, Add{}, shd);
        g2 = row_reduce<T>(g2, Add{}, shd) * 0x1p-40;
        const double k = st.r;
        double mx = 0.0;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const double z = __builtin_fma(g[j], (double)n, -g1) - f[j] * g2;
            g[j] = 4 * ((j / 4) * T + t) + j % 4 < n ? z * k : 0.0;
            mx = fmax(mx, fabs(g[j]));
        }
        const int scale = ey + gtop - ex;  // the row's results are g 2^scale
        if (p.mode == NORM_NEED) {
            if (ok) run = fmax(run, mx * pow2(scale));
            continue;
        }
        double in = inv * pow2(scale);
        if (p.mode == NORM_ROWS) {
            mx = row_reduce<T>(mx, Max{}, shd);
            const int need = need_f64(mx, p.q);
            int eo = need == NEED_NONE ? E_MIN : max(E_MIN, need + scale);
            if (ok && t == 0) {
                eo = clamp_exp_flag(eo, p.flags);
                p.oe[row] = (int8_t)eo;
            }
            in = pow2(scale - min(eo, E_MAX));
        }
        if (!ok) continue;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int c = 4 * (i * T + t);
            if (c < n)
                store4(p.out + off, c, n,
                       pack4(mant_of(g[4 * i], in), mant_of(g[4 * i + 1], in), mant_of(g[4 * i + 2], in),
                             mant_of(g[4 * i + 3], in)));
        }
    }
    if (grad && p.mode == NORM_NEED) {
        run = row_reduce<BT>(run, Max{}, shd);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = need_f64(run, p.q);
    }
    if (!sums) return;
    // the block's column sums: rows of one wave first, then the waves
    if constexpr (T < 64) {
#pragma unroll
        for (int j = 0; j < E; ++j)
#pragma unroll
            for (int s = T; s < 64; s <<= 1) {
                af[j] += __shfl_xor(af[j], s);
                ab[j] += __shfl_xor(ab[j], s);
            }
    }
    long long *pf = p.pf + (long long)blockIdx.x * n;
    int *pb = p.pb + (long long)blockIdx.x * n;
    if constexpr (T <= 64) {
        __shared__ double lf[4][T * E];
        __shared__ int lb[4][T * E];
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) < T) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                lf[wave][(j / 4 * T + t) * 4 + j % 4] = af[j];
                lb[wave][(j / 4 * T + t) * 4 + j % 4] = ab[j];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < n; c += BT) {
            pf[c] = (long long)(lf[0][c] + lf[1][c] + lf[2][c] + lf[3][c]);
            pb[c] = lb[0][c] + lb[1][c] + lb[2][c] + lb[3][c];
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int c = 4 * (j / 4 * T + t) + j % 4;
            if (c < n) {
                pf[c] = (long long)af[j];
                pb[c] = ab[j];
            }
        }
    }
}

#define IE_NORM_SHAPES(X) \
    X(16, 4) X(16, 8) X(16, 12) X(16, 16) X(32, 12) X(32, 16) X(64, 12) X(64, 16) X(256, 8) X(256, 12) X(256, 16) \
    X(1024, 8) X(1024, 12) X(1024, 16)

hipError_t launch_norm_fwd(const NormFwd &a, const NormPlan &pl, hipStream_t st) {
    prof_begin(st, PROF_NORM_FWD);
#define IE_CASE(T_, E_)                                                                                          \
    if (pl.t == T_ && pl.e == E_)                                                                                \
        hipLaunchKernelGGL((norm_fwd_kernel<T_, E_>), dim3(pl.grid), dim3(T_ > 256 ? T_ : 256), 0, st, a);
    IE_NORM_SHAPES(IE_CASE)
#undef IE_CASE
    prof_end(st, PROF_NORM_FWD);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwd &a, const NormPlan &pl, hipStream_t st) {
    prof_begin(st, PROF_NORM_BWD);
#define IE_CASE(T_, E_)                                                                                          \
    if (pl.t == T_ && pl.e == E_)                                                                                \
        hipLaunchKernelGGL((norm_bwd_kernel<T_, E_>), dim3(pl.grid), dim3(T_ > 256 ? T_ : 256), 0, st, a);
    IE_NORM_SHAPES(IE_CASE)
#undef IE_CASE
    prof_end(st, PROF_NORM_BWD);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Column sums
// ---------------------------------------------------------------------------

// Partial column sums of dY at its largest exponent: block (x, y) adds the
// rows [y chunk, (y + 1) chunk) of columns 256 x .. 256 x + 255, four columns
// per lane, every fourth row per wave.  |a| <= 128 and at most 2^23 rows a
// block keep the sums in 32 bits.
__global__ __launch_bounds__(256) void col_sum_kernel(const int8_t *dy, const int8_t *e, int e_row, const int *top,
                                                      long long rows, int cols, int chunk, int *pb) {
    __shared__ int sh[4][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 256 + lane * 4;
    const long long r0 = (long long)blockIdx.y * chunk, r1 = min(rows, r0 + chunk);
    const int dtop = top[0];
    int a[4] = {0, 0, 0, 0};
    if (c < cols)
        for (long long r = r0 + wave; r < r1; r += 4) {
            const uint32_t w = load4(dy + r * cols, c, cols);
            const int s = dtop - (int)e[e_row ? r : 0];
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] += rne_shift32(byte_of(w, k), s);
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) sh[wave][lane * 4 + k] = a[k];
    __syncthreads();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col < cols)
        pb[(long long)blockIdx.y * cols + col] =
            sh[0][threadIdx.x] + sh[1][threadIdx.x] + sh[2][threadIdx.x] + sh[3][threadIdx.x];
}

// Sums of `parts` partial rows (64-bit or 32-bit), 64 columns per block, at
// exponent base + *top: rounded into one group per channel here, or kept for
// col_round_kernel with the block's need.
__global__ __launch_bounds__(1024) void col_finish_kernel(ColOut f, ColOut b, int parts, int cols, const int *top,
                                                          uint32_t *flags) {
    __shared__ long long sh[16][64];
    const ColOut &o = blockIdx.y == 0 ? f : b;
    if (!o.m) return;
    const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    long long s = 0;
    if (c < cols) {
        if (o.p64)
            for (int i = grp; i < parts; i += 16) s += o.p64[(long long)i * cols + c];
        else
            for (int i = grp; i < parts; i += 16) s += o.p32[(long long)i * cols + c];
    }
    sh[grp][lane] = s;
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += sh[i][lane];
    const int eps = top[0] + o.base;
    int need = need64(s, eps, o.q);
    if (o.per) {
        if (c >= cols) return;
        const int e = clamp_exp_flag(max(E_MIN, need), flags);
        o.m[c] = (int8_t)rne_shift64(s, e - eps);
        o.e[c] = (int8_t)e;
        return;
    }
    need = wave_max_dpp(need);
    if (c < cols) o.sums[c] = s;
    if (lane == 0) o.need[blockIdx.x] = need;
}

// One exponent for the whole vector: every block takes the largest need.
__global__ __launch_bounds__(256) void col_round_kernel(ColOut f, ColOut b, int n_need, int cols, const int *top,
                                                        uint32_t *flags) {
    __shared__ int shi[4];
    const ColOut &o = blockIdx.y == 0 ? f : b;
    if (!o.m || o.per) return;
    int m = NEED_NONE;
    for (int i = threadIdx.x; i < n_need; i += 256) m = max(m, o.need[i]);
    m = row_reduce<256>(m, Max{}, shi);
    const int e = clamp_exp_flag(max(E_MIN, m), flags), s = e - top[0] - o.base;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < cols) o.m[c] = (int8_t)rne_shift64(o.sums[c], s);
    if (c == 0) o.e[0] = (int8_t)e;
}

hipError_t launch_col_sum(const int8_t *dy, const int8_t *e, int e_row, const int *top, long long rows, int cols,
                          int chunk, int parts, int *pb, hipStream_t st) {
    prof_begin(st, PROF_COL_SUM);
    hipLaunchKernelGGL(col_sum_kernel, dim3((cols + 255) / 256, parts), dim3(256), 0, st, dy, e, e_row, top, rows, cols,
                       chunk, pb);
    prof_end(st, PROF_COL_SUM);
    return hipGetLastError();
}

hipError_t launch_col_finish(const ColOut &f, const ColOut &b, int parts, int cols, const int *top, uint32_t *flags,
                             hipStream_t st) {
    const int nb = (cols + 63) / 64;
    prof_begin(st, PROF_COL_FINISH);
    hipLaunchKernelGGL(col_finish_kernel, dim3(nb, b.m ? 2 : 1), dim3(1024), 0, st, f, b, parts, cols, top, flags);
    if ((f.m && !f.per) || (b.m && !b.per))
        hipLaunchKernelGGL(col_round_kernel, dim3((cols + 255) / 256, b.m ? 2 : 1), dim3(256), 0, st, f, b, nb, cols,
                           top, flags);
    prof_end(st, PROF_COL_FINISH);
    return hipGetLastError();
}

}  // namespace ie
