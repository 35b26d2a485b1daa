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

// The statistics of a row held four mantissas to a word (zeros past its end).
// `sh` is another one than the row's before: threads may still read that.
template <int T, int W>
__device__ __forceinline__ RowStat row_stat(const uint32_t (&w)[W], int n, double n2eps, int eps_e, int e, int2 *sh) {
    int s = 0, q = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        s = __builtin_amdgcn_sdot4((int)w[i], 0x01010101, s, false);
        q = __builtin_amdgcn_sdot4((int)w[i], (int)w[i], q, false);
    }
    s = lane_reduce<(T < 64 ? T : 64)>(s, Add{});
    q = lane_reduce<(T < 64 ? T : 64)>(q, Add{});
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = make_int2(s, q);
        __syncthreads();
        s = q = 0;
#pragma unroll
        for (int i = 0; i < T / 64; ++i) {
            s += sh[i].x;
            q += sh[i].y;
        }
    }
    const double sd = (double)s, v = __builtin_fma((double)n, (double)q, -sd * sd);  // exact: below 2^43
    const double t = v + n2eps * pow2(eps_e - 2 * e);
    return RowStat{sd, t > 0.0 ? 1.0 / __builtin_sqrt(t) : 0.0};
}

// The values of four channels of a parameter vector from column c.
__device__ __forceinline__ void channel4(const NormVec &v, int c, int n, double absent, double (&o)[4]) {
    if (!v.m) {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = c + k < n ? absent : 0.0;
        return;
    }
    const uint32_t m = load4(v.m, c, n), e = v.per ? load4(v.e, c, n) : (uint32_t)(uint8_t)v.e[0] * 0x01010101u;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = (double)byte_of(m, k) * pow2(byte_of(e, k));
}

// The exponent of a whole-tensor result from the blocks' needs, by a block of
// BT threads; block 0 stores it.
template <int BT>
__device__ __forceinline__ int whole_exp(const int *bmax, int n, int8_t *oe, uint32_t *flags, int *sh) {
    int m = NEED_NONE;
    for (int i = threadIdx.x; i < n; i += BT) m = max(m, bmax[i]);
    m = row_reduce<BT>(m, Max{}, sh);
    const int e = clamp_exp_flag(max(E_MIN, m), flags);
    if (blockIdx.x == 0 && threadIdx.x == 0) oe[0] = (int8_t)e;
    return e;
}

template <int T>
constexpr int norm_block() {
    return T > 256 ? T : 256;
}

// T threads per row, E elements per thread.  gamma and beta stay in registers
// (E <= 12, or when a block holds one row) or in LDS; the next row's loads are
// in flight while a row is computed.
// Bound by instructions, 14 an element (issuing in 59 % of the cycles), and by
// the waits of two blocks a CU for loads and reductions (49 % of the waves'
// time), beside the stream: 25216 x 768 takes 14.7 us, 7.5 of them its 39 MB at
// the rate of a large copy; 4096 x 4096 17.2 us, 6.5.  A whole-tensor result
// reads X twice (25216 x 768: 24.7 us) unless one block holds it.
template <int T, int E, int BT>
__global__ __launch_bounds__(BT) void norm_fwd_kernel(NormFwd p) {
    using C = Cols<T, E>;
    constexpr int RPB = BT / T, W = E / 4;
    constexpr bool LDSV = T <= 64 && E > 12;
    __shared__ int2 sh2[2][BT / 64];
    __shared__ int shi[BT / 64], shm[BT / 64];
    __shared__ double2 gb[LDSV ? T * E : 1];
    const int t = threadIdx.x % T, slot = threadIdx.x / T, n = p.cols;
    const long long step = (long long)gridDim.x * RPB;
    C cols;
    cols.init(t, n);
    uint32_t w[W], next[W];
    int e = 0, e_next = 0;
    // the rows of a trip from r0; past the end: the last row again
    auto fetch = [&](long long r0) {
        const long long r = min(r0 + slot, p.rows - 1);
        cols.load(p.x + r * n, n % C::CH == 0 || r0 + RPB + C::CH <= p.rows, next);
        e_next = p.xe[p.x_row ? r : 0];
    };
    fetch((long long)blockIdx.x * RPB);
    double gam[LDSV ? 1 : E], bet[LDSV ? 1 : E];
    if constexpr (LDSV) {
        // element-major, so that a row's threads read neighbours
        for (int x = threadIdx.x; x < T * W; x += BT) {
            const int j = 4 * (x / T), tt = x % T;
            double g[4], b[4];
            channel4(p.gamma, C::col(j, tt), n, 1.0, g);
            channel4(p.beta, C::col(j, tt), n, 0.0, b);
#pragma unroll
            for (int k = 0; k < 4; ++k) gb[(j + k) * T + tt] = make_double2(g[k], b[k]);
        }
        __syncthreads();
    } else {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
            double g[4], b[4];
            channel4(p.gamma, cols.col(j), n, 1.0, g);
            channel4(p.beta, cols.col(j), n, 0.0, b);
#pragma unroll
            for (int k = 0; k < 4; ++k) gam[j + k] = g[k], bet[j + k] = b[k];
        }
    }
    double inv = 0.0;  // of a whole-tensor result
    if (p.mode == NORM_ROUND) inv = pow2(-whole_exp<BT>(p.bmax, p.n_bmax, p.oe, p.flags, shi));
    int run = 0;  // high word of the largest magnitude (NORM_NEED)
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += step) {
        const long long row = r0 + slot;
        const bool ok = row < p.rows;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = next[i];
        e = e_next;
        if (r0 + step < p.rows) fetch(r0 + step);
        if constexpr (LDSV) asm volatile("" ::: "memory");  // gamma and beta stay in LDS
        cols.clear(w);
        RowStat st;
        if (p.mode == NORM_ROUND) {
            st = p.stat[ok ? row : p.rows - 1];
        } else {
            st = row_stat<T>(w, n, p.n2eps, p.eps_e, e, sh2[turn ^= 1]);
            if (p.mode == NORM_NEED && ok && t == 0) p.stat[row] = st;
        }
        const float nf = (float)n, s128 = (float)st.s + 128.0f * nf;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] ^= 0x80808080u;
        double y[E];
        MaxMag mx;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const double d = centred(w[j / 4], j % 4, nf, s128);
            // past the row gamma and beta are zero, and so is y
            if constexpr (LDSV) {
                const double2 v = gb[j * T + t];
                y[j] = (d * st.r) * v.x + v.y;
            } else {
                y[j] = (d * st.r) * gam[j] + bet[j];
            }
            if (j % 2) mx.add(y[j - 1], y[j]);
        }
        if (p.mode == NORM_NEED) {
            run = max(run, mx.word());
            continue;
        }
        if (p.mode == NORM_ROWS) {
            int ex = max(E_MIN, need_word(row_reduce_once<T>(mx.word(), Max{}, shm), p.q));
            if (ok && t == 0) {
                ex = clamp_exp_flag(ex, p.flags);
                p.oe[row] = (int8_t)ex;
            }
            inv = pow2(-min(ex, E_MAX));
        }
        if (p.mode == NORM_ONE) {
            // the block holds the matrix (threads past the end a row again)
            const int ex = clamp_exp_flag(max(E_MIN, need_word(row_reduce<BT>(mx.word(), Max{}, shi), p.q)), p.flags);
            if (threadIdx.x == 0) p.oe[0] = (int8_t)ex;
            inv = pow2(-ex);
        }
        if (!ok) continue;
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i] = pack4(mant_of(y[4 * i], inv), mant_of(y[4 * i + 1], inv), mant_of(y[4 * i + 2], inv),
                         mant_of(y[4 * i + 3], inv));
        cols.store(p.out + row * n, w);
    }
    if (p.mode == NORM_NEED) {
        const int m = row_reduce<BT>(run, Max{}, shi);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = need_word(m, p.q);
    }
}

// A thread's share of the largest of n exponents, of BT threads; several loads
// in flight.
template <int BT>
__device__ __forceinline__ int max_exp_part(const int8_t *e, long long n) {
    int m = E_MIN;
    const long long whole = n / 16;
#pragma unroll 4
    for (long long c = threadIdx.x; c < whole; c += BT) {
        uint32_t w[4];
        __builtin_memcpy(w, e + 16 * c, 16);
#pragma unroll
        for (int k = 0; k < 16; ++k) m = max(m, byte_of(w[k / 4], k % 4));
    }
    const long long c = 16 * whole + threadIdx.x;
    return c < n ? max(m, (int)e[c]) : m;
}

// The same for the largest exponent of dY's rows: found by this block, or the
// largest of tops_kernel's.
template <int BT>
__device__ __forceinline__ int top_part(const int8_t *e, int e_row, long long rows, const int *tops, int n_tops) {
    if (!e_row) return e[0];
    if (!n_tops) return max_exp_part<BT>(e, rows);
    int m = E_MIN;
    for (int i = 0; i < n_tops; ++i) m = max(m, tops[i]);
    return m;
}

// Backward: NORM_NEED and NORM_ROWS also add up the columns of dgamma and
// dbeta (p.pf, p.pb: one row of partial sums per block).
// Bound by its instructions, 45 an element (62 % of the cycles issue one, 49 %
// where a row takes a block), and its waits (44 and 50 % of the waves' time: two waves a SIMD by the
// registers that hold the sums): 50432 x 192 takes 21 us and its sums' end 4,
// 5.6 of them its 29 MB at the rate of a large copy.  Wide rows, one to a block,
// add their partial sums' way through memory: 4096 x 4096 takes 45 us in all, 9.6
// of them X, dY and dX.
template <int T, int E>
__global__ __launch_bounds__(grad_block(T)) __attribute__((amdgpu_waves_per_eu(T > 512 ? 4 : 2)))
void norm_bwd_kernel(NormBwd p) {
    using C = Cols<T, E>;
    constexpr int BT = grad_block(T), RPB = BT / T, W = E / 4;
    constexpr bool LEAN = T > 512;  // 128 registers: g is made again where it is used
    __shared__ int2 sh2[2][BT / 64];
    __shared__ int shi[BT / 64], shm[BT / 64];
    __shared__ double shd[2][T > 64 ? BT / 64 : 1];
    const int t = threadIdx.x % T, slot = threadIdx.x / T, n = p.cols;
    const bool sums = p.pf && p.mode != NORM_ROUND, grad = p.out != nullptr;
    const long long step = (long long)gridDim.x * RPB;
    C cols;
    cols.init(t, n);
    uint32_t w[W], v[W], w_next[W], v_next[W];
    int ex = 0, ey = 0, ex_next = 0, ey_next = 0;
    auto fetch = [&](long long r0) {
        const long long r = min(r0 + slot, p.rows - 1);
        const bool whole = n % C::CH == 0 || r0 + RPB + C::CH <= p.rows;
        cols.load(p.x + r * n, whole, w_next);
        cols.load(p.dy + r * n, whole, v_next);
        ex_next = p.xe[p.x_row ? r : 0];
        ey_next = p.dye[p.dy_row ? r : 0];
    };
    fetch((long long)blockIdx.x * RPB);
    // the largest exponents of dY and of gamma's channels, gamma's loads ahead of them
    uint32_t gw[W], ge[W];
    if (p.gamma.m) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            gw[i] = load4(p.gamma.m, cols.col(4 * i), n);
            ge[i] = p.gamma.per ? load4(p.gamma.e, cols.col(4 * i), n) : 0u;
        }
    }
    int2 top = make_int2(sums ? top_part<BT>(p.dye, p.dy_row, p.rows, p.tops, p.n_tops) : E_MIN,
                         !p.gamma.m ? 0 : p.gamma.per ? max_exp_part<BT>(p.gamma.e, n) : p.gamma.e[0]);
    top.x = lane_reduce<64>(top.x, Max{});
    top.y = lane_reduce<64>(top.y, Max{});
    if ((threadIdx.x & 63) == 0) sh2[0][threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < BT / 64; ++i) {
        top.x = max(top.x, sh2[0][i].x);
        top.y = max(top.y, sh2[0][i].y);
    }
    const int dtop = top.x, gtop = top.y;
    if (sums && blockIdx.x == 0 && threadIdx.x == 0) *p.top = dtop;
    // gamma re-expressed, four mantissas to a word
    double gam[LEAN ? 1 : E];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (!p.gamma.m) {
            gw[i] = 0x01010101u & cols.mask[i];
        } else if (p.gamma.per) {
            const uint32_t m = gw[i], e = ge[i];
            gw[i] = pack4(rne_shift32(byte_of(m, 0), gtop - byte_of(e, 0)), rne_shift32(byte_of(m, 1), gtop - byte_of(e, 1)),
                          rne_shift32(byte_of(m, 2), gtop - byte_of(e, 2)), rne_shift32(byte_of(m, 3), gtop - byte_of(e, 3)));
        }
        if constexpr (!LEAN) {
#pragma unroll
            for (int k = 0; k < 4; ++k) gam[4 * i + k] = (double)byte_of(gw[i], k);
        }
    }
    double inv = 0.0;
    if (p.mode == NORM_ROUND) inv = pow2(-whole_exp<BT>(p.bmax, p.n_bmax, p.oe, p.flags, shi));
    double af[E];
    int ab[E];
#pragma unroll
    for (int j = 0; j < E; ++j) af[j] = 0.0, ab[j] = 0;
    int run = 0;  // high word of the largest magnitude (NORM_NEED)
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += step) {
        const long long row = r0 + slot;
        const bool ok = row < p.rows;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = w_next[i], v[i] = v_next[i];
        ex = ex_next;
        ey = ey_next;
        if (r0 + step < p.rows) fetch(r0 + step);
        cols.clear(w);
        cols.clear(v);
        GradStat gs;
        if (p.mode == NORM_ROUND) {
            gs = p.gstat[ok ? row : p.rows - 1];
        } else {
            const RowStat st = row_stat<T>(w, n, p.n2eps, p.eps_e, ex, sh2[turn ^= 1]);
            gs.s = st.s;
            gs.r = st.r;
        }
        const double r20 = gs.r * 1048576.0;  // h 2^20 = d (r 2^20)
        // a = dY at its largest exponent: rows past the end count for nothing
        const double as = ok ? pow2(max(ey - dtop, -64)) : 0.0;
        const float nf = (float)n, s128 = (float)gs.s + 128.0f * nf;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] ^= 0x80808080u;
        double f[E], g[LEAN ? 1 : E], g2 = 0.0;
        auto g_of = [&](int j) { return (double)byte_of(v[j / 4], j % 4) * (LEAN ? (double)byte_of(gw[j / 4], j % 4) : gam[LEAN ? 0 : j]); };
        int g1 = 0;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const double d = centred(w[j / 4], j % 4, nf, s128);
            const double c = (double)byte_of(v[j / 4], j % 4);
            f[j] = __builtin_rint(d * r20);
            if constexpr (!LEAN) g[j] = c * gam[j];
            if (sums) {
                const double a = __builtin_fma(c, as, ROUND_MAGIC);
                af[j] = __builtin_fma(a - ROUND_MAGIC, f[j], af[j]);
                ab[j] += __double2loint(a);
            }
        }
        if (!grad) continue;
        auto forget = [&] {  // nothing made of these words before is kept
            if constexpr (LEAN) {
#pragma unroll
                for (int i = 0; i < W; ++i) asm volatile("" : "+v"(v[i]), "+v"(gw[i]));
            }
        };
        forget();
        if (p.mode != NORM_ROUND) {
#pragma unroll
            for (int i = 0; i < W; ++i) g1 = __builtin_amdgcn_sdot4((int)v[i], (int)gw[i], g1, false);
#pragma unroll
            for (int j = 0; j < E; ++j) g2 = __builtin_fma(LEAN ? g_of(j) : g[LEAN ? 0 : j], f[j], g2);
            g1 = lane_reduce<(T < 64 ? T : 64)>(g1, Add{});
            g2 = lane_reduce<(T < 64 ? T : 64)>(g2, Add{});
            gs.g1 = (double)g1;
            if constexpr (T > 64) {
                if ((threadIdx.x & 63) == 0) shd[0][threadIdx.x >> 6] = gs.g1, shd[1][threadIdx.x >> 6] = g2;
                __syncthreads();
                gs.g1 = g2 = 0.0;
#pragma unroll
                for (int i = 0; i < T / 64; ++i) gs.g1 += shd[0][i], g2 += shd[1][i];
            }
            gs.g2 = g2 * 0x1p-40;
            if (p.mode == NORM_NEED && ok && t == 0) p.gstat[row] = gs;
        }
        forget();
#pragma unroll
        for (int j = 0; j < E; ++j) {
            // the result takes f's place
            f[j] = (__builtin_fma(LEAN ? g_of(j) : g[LEAN ? 0 : j], (double)n, -gs.g1) - f[j] * gs.g2) * gs.r;
        }
        if (!cols.exact) {
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (!(cols.mask[j / 4] >> (8 * (j % 4)) & 1u)) f[j] = 0.0;
        }
        MaxMag mx;
#pragma unroll
        for (int j = 0; j < E; j += 2) mx.add(f[j], f[j + 1]);
        const int scale = ey + gtop - ex;  // the row's results are f 2^scale
        if (p.mode == NORM_NEED) {
            if (mx.word()) run = max(run, mx.word() + (scale << 20));
            continue;
        }
        if (p.mode == NORM_ONE) {
            const int m = row_reduce<BT>(mx.word() ? mx.word() + (scale << 20) : 0, Max{}, shi);
            const int eo = clamp_exp_flag(max(E_MIN, need_word(m, p.q)), p.flags);
            if (threadIdx.x == 0) p.oe[0] = (int8_t)eo;
            inv = pow2(-eo);
        }
        double in = inv * pow2(scale);
        if (p.mode == NORM_ROWS) {
            const int need = need_word(row_reduce_once<T>(mx.word(), Max{}, shm), p.q);
            int eo = need == NEED_NONE ? E_MIN : max(E_MIN, need + scale);
            if (ok && t == 0) {
                eo = clamp_exp_flag(eo, p.flags);
                p.oe[row] = (int8_t)eo;
            }
            in = pow2(scale - min(eo, E_MAX));
        }
        if (!ok) continue;
#pragma unroll
        for (int i = 0; i < W; ++i)
            w[i] = pack4(mant_of(f[4 * i], in), mant_of(f[4 * i + 1], in), mant_of(f[4 * i + 2], in),
                         mant_of(f[4 * i + 3], in));
        cols.store(p.out + row * n, w);
    }
    if (grad && p.mode == NORM_NEED) {
        run = row_reduce<BT>(run, Max{}, shi);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = need_word(run, p.q);
    }
    if (!sums) return;
    // the block's column sums (a's low words carry nothing of ROUND_MAGIC)
    const int np = col_pitch(n);
    long long *pf = p.pf + (long long)blockIdx.x * np;
    int *pb = p.pb + (long long)blockIdx.x * np;
    auto put = [&](int c, const double (&a)[4]) {
        *(longlong2 *)(pf + c) = longlong2{(long long)a[0], (long long)a[1]};
        *(longlong2 *)(pf + c + 2) = longlong2{(long long)a[2], (long long)a[3]};
    };
    if constexpr (T > 64) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int c = cols.col(4 * i);
            if (c >= n) continue;
            put(c, {af[4 * i], af[4 * i + 1], af[4 * i + 2], af[4 * i + 3]});
            *(v4i *)(pb + c) = v4i{ab[4 * i], ab[4 * i + 1], ab[4 * i + 2], ab[4 * i + 3]};
        }
    } else {
        // the waves' sums meet in LDS, dgamma's and then dbeta's
        __shared__ double sums_lds[BT / 64][T * E];
        const int wave = threadIdx.x >> 6;
        const bool mine = (threadIdx.x & 63) < T;
        int(*ib)[T * E] = (int(*)[T * E])sums_lds;
        auto rows_of_wave = [](auto a) {
            if constexpr (T <= 16) a = swap_reduce<16>(a, Add{});
            if constexpr (T <= 32) a = swap_reduce<32>(a, Add{});
            return a;
        };
        // element j of thread c / CH % T holds column c
        auto place = [](int c) { return (c / (C::CH * T) * C::CH + c % C::CH) * T + c / C::CH % T; };
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const double a = rows_of_wave(af[j]);
            if (mine) sums_lds[wave][j * T + t] = a;
        }
        __syncthreads();
        for (int c = 4 * threadIdx.x; c < n; c += 4 * BT) {
            double a[4] = {0.0, 0.0, 0.0, 0.0};
            const int at = place(c);
#pragma unroll
            for (int i = 0; i < BT / 64; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) a[k] += sums_lds[i][at + k * T];
            put(c, a);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int a = rows_of_wave(ab[j]);
            if (mine) ib[wave][j * T + t] = a;
        }
        __syncthreads();
        for (int c = 4 * threadIdx.x; c < n; c += 4 * BT) {
            v4i a = {0, 0, 0, 0};
            const int at = place(c);
#pragma unroll
            for (int i = 0; i < BT / 64; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) a[k] += ib[i][at + k * T];
            *(v4i *)(pb + c) = a;
        }
    }
}

// Largest exponents of runs of rows, one per block, for matrices too tall for
// every block of norm_bwd_kernel to find the largest itself.
__global__ __launch_bounds__(1024) void tops_kernel(const int8_t *e, long long n, long long run, int *tops) {
    __shared__ int shi[16];
    const long long b = blockIdx.x * run;
    const int m = row_reduce<1024>(max_exp_part<1024>(e + b, min(run, n - b)), Max{}, shi);
    if (threadIdx.x == 0) tops[blockIdx.x] = m;
}

hipError_t launch_norm_fwd(const NormFwd &a, const NormPlan &pl, hipStream_t st) {
    if (!(a.mode == NORM_ONE ? norm_one_built(pl) : norm_fwd_built(pl))) return hipErrorInvalidValue;
    prof_begin(st, PROF_NORM_FWD);
#define IE_CASE(T_, E_)           \
    if (pl.t == T_ && pl.e == E_) \
        hipLaunchKernelGGL((norm_fwd_kernel<T_, E_, norm_block<T_>()>), dim3(pl.grid), dim3(norm_block<T_>()), 0, st, a);
#define IE_ONE(T_, E_)            \
    if (pl.t == T_ && pl.e == E_) hipLaunchKernelGGL((norm_fwd_kernel<T_, E_, 1024>), dim3(1), dim3(1024), 0, st, a);
    if (a.mode == NORM_ONE) {
        IE_NORM_ONE(IE_ONE)
    } else {
        IE_NORM_FWD(IE_CASE)
    }
#undef IE_CASE
#undef IE_ONE
    prof_end(st, PROF_NORM_FWD);
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwd &a, const NormPlan &pl, hipStream_t st) {
    if (!norm_bwd_built(pl)) return hipErrorInvalidValue;
    prof_begin(st, PROF_NORM_BWD);
#define IE_CASE(T_, E_)       \
    if (pl.t == T_ && pl.e == E_) \
        hipLaunchKernelGGL((norm_bwd_kernel<T_, E_>), dim3(pl.grid), dim3(grad_block(T_)), 0, st, a);
    IE_NORM_BWD(IE_CASE)
#undef IE_CASE
    prof_end(st, PROF_NORM_BWD);
    return hipGetLastError();
}

hipError_t launch_tops(const int8_t *e, long long n, int *tops, int n_tops, hipStream_t st) {
    const long long run = (n + n_tops - 1) / n_tops;
    hipLaunchKernelGGL(tops_kernel, dim3((int)((n + run - 1) / run)), dim3(1024), 0, st, e, n, run, tops);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Column sums
// ---------------------------------------------------------------------------

// Partial column sums of dY at its largest exponent: block (x, y) adds the
// rows [y chunk, (y + 1) chunk) of columns 256 x .. 256 x + 255, 16 columns
// per thread, four rows to a wave, four loads in flight.
// A mantissa at shift s <= 7 is one conversion (of C + 128, unsigned) and one
// fp32 fused multiply-add, exact before its only rounding, whose low bits are
// the rounded integer above those of 1.5 * 2^23; these are summed as they
// are and the constant taken off at the end (modulo 2^32).  At s >= 8 every
// |C| <= 128 rounds to 0.  At most 2^23 rows a block keep a sum in 32 bits.
// Bound by its instructions, six an element (70 % of the cycles issue one):
// 25216 x 2304 takes 14.2 us, 11 of them its 58 MB at the rate of a large copy.
__global__ __launch_bounds__(256) void col_sum_kernel(const int8_t *dy, const int8_t *e, int e_row, long long rows,
                                                      int cols, int chunk, const int *tops, int n_tops, int *top,
                                                      int *pb) {
    constexpr int U = 4, RPT = 16;  // rows of a block's trip: a thread takes every 16th
    __shared__ uint32_t sh[4][256];
    __shared__ int shi[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, slot = threadIdx.x >> 4;
    const int c = blockIdx.x * 256 + (lane & 15) * 16;
    const long long r0 = (long long)blockIdx.y * chunk, r1 = min(rows, r0 + chunk);
    const int dtop = row_reduce<256>(top_part<256>(e, e_row, rows, tops, n_tops), Max{}, shi);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *top = dtop;
    // 16 bytes may be read past a row's end wherever as many more rows follow;
    // sums of columns past the last are not kept
    const bool whole = cols % 16 == 0 || r1 + 16 <= rows;
    const int c0 = c < cols ? c : 0;
    uint32_t a[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) a[k] = 0;
    uint32_t n_add = 0;
    for (long long r = r0 + slot; r < r1; r += RPT * U) {
        uint32_t w[U][4];
        int s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long rr = min(r + RPT * u, r1 - 1);  // past the end: a row that counts for nothing
            if (whole) __builtin_memcpy(w[u], dy + rr * cols + c0, 16);
            else load_run<16>(dy + rr * cols, c, cols, w[u]);
            s[u] = e[e_row ? rr : 0];
        }
        n_add += U;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int sh = r + RPT * u < r1 ? dtop - s[u] : 8;
            const float f = sh < 8 ? __builtin_ldexpf(1.0f, -sh) : 0.0f, k0 = 12582912.0f - 128.0f * f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint32_t x = w[u][k / 4] ^ 0x80808080u;
                a[k] += (uint32_t)__float_as_int(__builtin_fmaf((float)(x >> (8 * (k % 4)) & 255u), f, k0));
            }
        }
    }
    // every addition brought the constant along
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        int v = (int)(a[k] - n_add * 0x4B400000u);
        v = swap_reduce<32>(swap_reduce<16>(v, Add{}), Add{});
        if (lane < 16) sh[wave][lane * 16 + k] = (uint32_t)v;
    }
    __syncthreads();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col < cols)
        pb[(long long)blockIdx.y * col_pitch(cols) + col] =
            (int)(sh[0][threadIdx.x] + sh[1][threadIdx.x] + sh[2][threadIdx.x] + sh[3][threadIdx.x]);
}

// Sums of `parts` partial rows (64-bit or 32-bit), 16 columns at a time per block
// and 64 partial rows at a time, at exponent base + *top: rounded into one group per
// channel here, or kept for col_round_kernel with the block's need.  TURNS: the
// blocks take turns, over vectors of 2^20 channels and more (narrower ones do
// without the barrier between turns: 100 x 524288 120 us, 135 with it).
template <bool TURNS>
__global__ __launch_bounds__(1024) void col_finish_kernel(ColOut f, ColOut b, int parts, int cols, const int *top,
                                                          uint32_t *flags) {
    __shared__ long long sh[16][16];
    const ColOut &o = blockIdx.y == 0 ? f : b;
    if (!o.m) return;
    const int lane = threadIdx.x & 15, grp = threadIdx.x >> 4, eps = top[0] + o.base;
    const long long pitch = col_pitch(cols);
    int block_need = NEED_NONE;
    for (long long c = blockIdx.x * 16ll + lane; c - lane < cols; c += gridDim.x * 16ll) {
        long long s = 0;
        if (c < cols) {
            if (o.p64) {
#pragma unroll 4
                for (int i = grp; i < parts; i += 64) s += o.p64[(long long)i * pitch + c];
            } else {
#pragma unroll 4
                for (int i = grp; i < parts; i += 64) s += o.p32[(long long)i * pitch + c];
            }
        }
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if ((threadIdx.x & 63) < 16) sh[threadIdx.x >> 6][lane] = s;
        __syncthreads();
        if (threadIdx.x < 64) {
            s = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) s += sh[i][lane];
            const int need = c < cols ? need64(s, eps, o.q) : NEED_NONE;
            if (threadIdx.x < 16 && c < cols) {
                if (o.per) {
                    const int e = clamp_exp_flag(max(E_MIN, need), flags);
                    o.m[c] = (int8_t)rne_shift64(s, e - eps);
                    o.e[c] = (int8_t)e;
                } else {
                    o.sums[c] = s;
                }
            }
            block_need = max(block_need, need);
        }
        if constexpr (!TURNS) break;
        __syncthreads();  // the sums are read
    }
    if (!o.per && threadIdx.x < 64) {
        block_need = lane_reduce<16>(block_need, Max{});
        if (threadIdx.x == 0) o.need[blockIdx.x] = block_need;
    }
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
    for (int c = blockIdx.x * 256 + threadIdx.x; c < cols; c += gridDim.x * 256) o.m[c] = (int8_t)rne_shift64(o.sums[c], s);
    if (blockIdx.x == 0 && threadIdx.x == 0) o.e[0] = (int8_t)e;
}

// The same in one launch for a few short partial rows (parts <= COL_FEW, cols
// <= 4096): a block per vector.
__global__ __launch_bounds__(1024) void col_few_kernel(ColOut f, ColOut b, int parts, int cols, const int *top,
                                                       uint32_t *flags) {
    __shared__ int shi[16];
    const ColOut &o = blockIdx.y == 0 ? f : b;
    if (!o.m) return;
    const int pitch = col_pitch(cols), eps = top[0] + o.base;
    long long s[4] = {0, 0, 0, 0};
    int need[4], m = NEED_NONE;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = threadIdx.x + 1024 * k;
        if (c < cols) {
#pragma unroll 4
            for (int i = 0; i < parts; ++i) s[k] += o.p64 ? o.p64[i * pitch + c] : (long long)o.p32[i * pitch + c];
        }
        need[k] = c < cols ? need64(s[k], eps, o.q) : NEED_NONE;
        m = max(m, need[k]);
    }
    if (!o.per) m = row_reduce<1024>(m, Max{}, shi);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = threadIdx.x + 1024 * k;
        if (c >= cols) continue;
        const int e = clamp_exp_flag(max(E_MIN, o.per ? need[k] : m), flags);
        o.m[c] = (int8_t)rne_shift64(s[k], e - eps);
        if (o.per || c == 0) o.e[c] = (int8_t)e;
    }
}

hipError_t launch_col_sum(const int8_t *dy, const int8_t *e, int e_row, long long rows, int cols, ColPlan pl,
                          const int *tops, int n_tops, int *top, int *pb, hipStream_t st) {
    prof_begin(st, PROF_COL_SUM);
    hipLaunchKernelGGL(col_sum_kernel, dim3((cols + 255) / 256, pl.parts), dim3(256), 0, st, dy, e, e_row, rows, cols,
                       pl.chunk, tops, n_tops, top, pb);
    prof_end(st, PROF_COL_SUM);
    return hipGetLastError();
}

hipError_t launch_col_finish(const ColOut &f, const ColOut &b, int parts, int cols, const int *top, uint32_t *flags,
                             hipStream_t st) {
    const int nb = col_blocks(cols);
    const bool whole = (f.m && !f.per) || (b.m && !b.per);
    prof_begin(st, PROF_COL_FINISH);
    if (whole && parts <= COL_FEW && cols <= 4096) {
        hipLaunchKernelGGL(col_few_kernel, dim3(1, b.m ? 2 : 1), dim3(1024), 0, st, f, b, parts, cols, top, flags);
        prof_end(st, PROF_COL_FINISH);
        return hipGetLastError();
    }
    const dim3 grid(nb, b.m ? 2 : 1), block(1024);
    if (nb < COL_BLOCKS) hipLaunchKernelGGL(col_finish_kernel<false>, grid, block, 0, st, f, b, parts, cols, top, flags);
    else hipLaunchKernelGGL(col_finish_kernel<true>, grid, block, 0, st, f, b, parts, cols, top, flags);
    if (whole) {
        const int g = (cols + 255) / 256;
        hipLaunchKernelGGL(col_round_kernel, dim3(g < 1024 ? g : 1024, b.m ? 2 : 1), dim3(256), 0, st, f, b, nb, cols,
                           top, flags);
    }
    prof_end(st, PROF_COL_FINISH);
    return hipGetLastError();
}

}  // namespace ie
