// Forward product with bias, residual and ReLU whose result rows lie whole
// inside a workgroup, so that a row's exponent is known before it leaves the
// registers: one pass, no intermediate result in memory.
//
// A workgroup of 8 waves computes 64 rows and 256 NI >= N columns at a time
// (NI <= 2: two of 4 waves share the CU with 32 rows each, one's epilogue beside
// the other's products; wider rows would stream too much weight that way), each
// wave an equal share of the columns of every row, with
// v_mfma_i32_32x32x32_i8 run transposed (a lane holds one row of the result).
// The weight is laid out beforehand in the order the matrix instructions take
// it (1 KiB for 32 rows and 32 contraction bytes, lane by lane), so a wave
// streams its share of it from L2 straight into registers, two steps ahead;
// the rows of X are staged in LDS, up to 1024 contraction bytes at a time.
// Nothing in the contraction loop waits for another wave.
// Workgroups are persistent: the next tile's X is loaded during the products
// (a long one's, and the residual, while the result is stored, when the
// registers are free), after one word of each of its lines has brought it into
// L2.
//
// The epilogue holds y in fp64, in the registers the accumulators leave, so
// each value is computed once (NI = 4 has no room and computes it twice).
//
// Bound by its phases one after the other: over 50432 x 768 x 192 the cycles
// are 48 % fp64 and conversion instructions of the epilogue, 42 % LDS (column
// scales and biases, staging) and 14 % products (25216 x 768 x 768: 32, 32 and
// 23 %), and the registers hold no second workgroup of NI >= 3 to set beside.
// Measured, with the weight's layout (3 to 5 us), from box to box: 50432 x 768 x
// 192 31 to 34 us, 45 to 47 with a residual (round to odd by tiles and the pass
// that closes it: 74 without), 25216 x 768 x 768 with a residual 37 to 41 us (51).
#include <algorithm>
#include <type_traits>

#include "ie_f64.h"
#include "ie_internal.h"

#pragma clang fp contract(off)

namespace ie {

// W [N x K] -> out[n / 32][k / 32][lane][16], lane l holding row l % 32 and
// bytes 16 (l / 32) .. + 15 of the 32; zeros past N and K.  A block lays out
// 32 rows and 128 contraction bytes.
__global__ __launch_bounds__(256) void tile_weight_kernel(const int8_t *w, int N, int K, int ks, int8_t *out) {
    const int row = threadIdx.x >> 3, c = threadIdx.x & 7;
    const int n = blockIdx.x * 32 + row, k = blockIdx.y * 128 + 16 * c, step = k >> 5;
    uint32_t v[4] = {0, 0, 0, 0};
    if (step >= ks) return;
    if (n < N) load_run<16>(w + (long long)n * K, k, K, v);
    *(v4i *)(out + (((long long)blockIdx.x * ks + step) * 64 + (c & 1) * 32 + row) * 16) =
        v4i{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}

// KC: contraction steps of X in LDS.  RES: no residual, one with 16-byte aligned
// rows, any other.
enum { RES_NONE, RES_VEC, RES_ANY };
template <int NI, int KC, int RES>
struct RowsCfg {
    static constexpr int BN = 256 * NI, RP = BN + 16;  // RP: pitch of the residual / result tile
    // blocks of 32 rows, waves, and a wave's blocks of 32 columns
    static constexpr int MA = NI <= 2 ? 1 : 2, WV = 4 * MA, NB = 8 * NI / WV, BM = 32 * MA, THR = 64 * WV;
    static constexpr int PER_CU = NI == 1 ? 4 : NI == 2 ? 2 : 1;  // resident workgroups
    static constexpr int D = 2;  // steps of the weight in flight
    static constexpr bool KEEP = NI < 4;
    static constexpr bool AHEAD = NI < 4 || RES == RES_NONE;  // room for a second quad's terms
    // the next tile's X is loaded during the products where it fits the registers
    static constexpr bool EARLY = KC <= 8 && (RES == RES_NONE || NI <= 2);
    static constexpr int A = KC * 1024 * MA, CS = A + 16 * BN, RED = CS + WV * BM * 4, LDS = RED + BM * RP;
};

template <int NI, int KC, int RES>
__global__ __launch_bounds__((RowsCfg<NI, KC, RES>::THR)) __attribute__((amdgpu_waves_per_eu(NI == 1 ? 4 : 2)))
void rows_add_kernel(const int8_t *x, const int8_t *wt, int M, int N, int K, int ks, AddEpi e) {
    using C = RowsCfg<NI, KC, RES>;
    constexpr int BN = C::BN, RP = C::RP, D = C::D, U = KC / 4, MA = C::MA, NB = C::NB, WV = C::WV;
    constexpr int BM = C::BM, THR = C::THR;
    __shared__ __attribute__((aligned(16))) int8_t lds[C::LDS];
    double *cs = (double *)(lds + C::A), *bs = cs + BN;  // column scales, bias
    int *red = (int *)(lds + C::CS);                    // row maxima of the waves [WV][BM]
    int8_t *rt = lds + C::RED;                          // the residual, then the result
    int tid = threadIdx.x;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles = (M + BM - 1) / BM;

    // X: thread t takes, of row (t / 4) % 64, the 16-byte piece t % 4 + 4 (t / 256)
    // of every four contraction steps; rows past the last repeat it, bytes past K
    // (the next row's) meet zeros of the weight, and at the matrix's end its last
    // 16 bytes are moved down
    auto fetch_x = [&](int tile, int s0, v4i (&an)[U]) {
        const int arow = (tid >> 2) & (BM - 1), aj = (tid & 3) + 4 * (tid / (4 * BM));
        const long long o = (long long)min(tile * BM + arow, M - 1) * K, last = (long long)M * K - 16;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s0 + 4 * u) * 32 + aj * 16;
            const long long p = o + (k < K ? k : 0), over = p - last;
            uint64_t v[2];
            __builtin_memcpy(v, x + min(p, last), 16);
            if (over > 0) {
                const int s = 8 * (int)over;
                v[0] = s < 64 ? v[0] >> s | v[1] << (64 - s) : v[1] >> (s - 64);
                v[1] = s < 64 ? v[1] >> s : 0;
            }
            an[u] = v4i{(int)v[0], (int)(v[0] >> 32), (int)v[1], (int)(v[1] >> 32)};
        }
    };
    auto store_x = [&](const v4i (&an)[U]) {
        const int arow = (tid >> 2) & (BM - 1), aj = (tid & 3) + 4 * (tid / (4 * BM));
        int8_t *ad = lds + (((aj >> 1) * MA + (arow >> 5)) * 64 + (aj & 1) * 32 + (arow & 31)) * 16;
#pragma unroll
        for (int u = 0; u < U; ++u) *(v4i *)(ad + u * 4096 * MA) = an[u];
    };
    // the residual of a tile, 16 bytes at a time
    // (16 threads a row, every 16th piece each)
    constexpr int RPP = THR / 16, RR = BM / RPP * NI;  // rows of a pass, pieces of a thread
    auto fetch_r = [&](int tile, v4i (&rr)[RR]) {
        if constexpr (RES == RES_NONE) return;
#pragma unroll
        for (int i = 0; i < RR; ++i) {
            const int row = i / NI * RPP + (tid >> 4), c = ((tid & 15) + 16 * (i % NI)) * 16;
            const int8_t *src = e.r + (long long)min(tile * BM + row, M - 1) * N;
            if constexpr (RES == RES_VEC) {
                rr[i] = *(const v4i *)(src + (c < N ? c : 0));
            } else {
                rr[i] = load16(src, min(c, N - 1), N);
            }
        }
    };
    auto store_r = [&](const v4i (&rr)[RR]) {
        if constexpr (RES != RES_NONE) {
#pragma unroll
            for (int i = 0; i < RR; ++i) {
                const int row = i / NI * RPP + (tid >> 4), c = ((tid & 15) + 16 * (i % NI)) * 16;
                *(v4i *)(rt + row * RP + c) = c < N ? rr[i] : v4i{0, 0, 0, 0};
            }
        }
    };
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(wt + (long long)wave * NB * ks * 1024), (short)0, NB * ks * 1024, 0x00020000);
    auto wtile = [&](int b, int s) -> v4i {
        return (v4i)__builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16, (b * ks + s) * 1024, 0);
    };

    v4i x0[U], r0[RR];
    fetch_x(blockIdx.x, 0, x0);
    fetch_r(blockIdx.x, r0);
    for (int n = tid; n < BN; n += THR) {
        // past the last column everything is zero
        cs[n] = n < N ? pow2((int)e.we[e.w_row ? n : 0]) : 0.0;
        bs[n] = n < N && e.bias.m ? (double)e.bias.m[n] * pow2((int)e.bias.e[e.bias.per ? n : 0]) : 0.0;
    }
    store_x(x0);
    store_r(r0);

    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int m0 = tile * BM, next = min(tile + (int)gridDim.x, tiles - 1);  // past the end: fetched, never used
        v4i xn[U], rn[RR];
        // offsets made of the thread's number are made anew for every tile: kept,
        // they would not fit the registers
        asm volatile("" : "+v"(tid));
        // one word of every 128 bytes of the next tile's rows, so that they are in L2
        // when they are fetched
        const int ahead = min(tile + (int)gridDim.x, tiles - 1) * BM + (tid >> 3);
        const long long arow = min(ahead, M - 1);
        uint32_t warm = 0;
        for (int c = (tid & 7) * 128; c < min(K - 3, KC * 32); c += 1024) warm |= *(const uint32_t *)(x + arow * K + c);
        if constexpr (RES == RES_VEC)
            for (int c = (tid & 7) * 128; c < N; c += 1024) warm |= *(const uint32_t *)(e.r + arow * N + c);
        // this lane's two rows' exponents
        double sx[MA], sr[MA];
#pragma unroll
        for (int a = 0; a < MA; ++a) {
            const int m = min(m0 + a * 32 + (lane & 31), M - 1);
            sx[a] = pow2((int)e.xe[e.x_row ? m : 0]);
            sr[a] = RES ? pow2((int)e.re[e.r_row ? m : 0]) : 0.0;
        }
        v16i acc[MA][NB];
        v4i bf[D][NB];
#pragma unroll
        for (int u = 0; u < D; ++u)
#pragma unroll
            for (int b = 0; b < NB; ++b) bf[u][b] = wtile(b, u);
        __syncthreads();  // X and the residual are there
        if constexpr (C::EARLY) fetch_x(next, 0, xn);

        const v4i *as = (const v4i *)lds + lane;
        // D steps from step s of the staged ones, k of the contraction; the very first
        // products start the sums
        auto go = [&](int s, int k, auto start) {
#pragma unroll
            for (int u = 0; u < D; ++u) {
                v4i af[MA];
#pragma unroll
                for (int a = 0; a < MA; ++a) af[a] = as[((s + u) * MA + a) * 64];
                const int next = min(k + u + D, ks - 1);  // past the end: loaded, never used
#pragma unroll
                for (int b = 0; b < NB; ++b) {
#pragma unroll
                    for (int a = 0; a < MA; ++a) {
                        if constexpr (decltype(start)::value) {
                            const v16i zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
                            acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[u][b], af[a], u ? acc[a][b] : zero, 0, 0, 0);
                        } else {
                            acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(bf[u][b], af[a], acc[a][b], 0, 0, 0);
                        }
                    }
                    bf[u][b] = wtile(b, next);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        go(0, 0, std::true_type{});
        for (int s0 = 0; s0 < ks; s0 += KC) {
            if (s0) {
                v4i an[U];
                fetch_x(tile, s0, an);
                __syncthreads();
                store_x(an);
                __syncthreads();
            }
            const int steps = min(KC, ks - s0);  // a multiple of D
            for (int s = s0 ? 0 : D; s < steps; s += D) go(s, s0 + s, std::false_type{});
        }
        asm volatile("" ::"v"(warm));
        __syncthreads();  // X is free

        // four neighbours of the result (columns 32 b + 8 h of this lane's own on) of
        // both rows this lane holds; each fused step is an exact product and one
        // rounded sum
        const int c0 = wave * 32 * NB + 4 * (lane >> 5);
        int ocs = C::A + 8 * c0, ort = C::RED + (lane & 31) * RP + c0;  // of its scales and residuals in LDS
        asm volatile("" : "+v"(ocs), "+v"(ort));
        // a quad's scales, biases and residuals, read while the one before is computed
        struct Terms {
            double s[4], o[4];
            uint32_t r[MA];
        };
        auto terms = [&](int q, Terms &t) {
            const double *s = (const double *)(lds + ocs) + 8 * q;
#pragma unroll
            for (int k = 0; k < 4; ++k) t.s[k] = s[k], t.o[k] = s[BN + k];
            if constexpr (RES) {
#pragma unroll
                for (int a = 0; a < MA; ++a) t.r[a] = *(const uint32_t *)(lds + ort + a * 32 * RP + 8 * q);
            }
        };
        auto quad = [&](int q, const Terms &t, double (&y)[MA][4]) {
#pragma unroll
            for (int a = 0; a < MA; ++a) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[a][k] = __builtin_fma((double)acc[a][q / 4][4 * (q % 4) + k], sx[a] * t.s[k], t.o[k]);
                if constexpr (RES) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[a][k] = __builtin_fma((double)byte_of(t.r[a], k), sr[a], y[a][k]);
                }
            }
        };
        double yk[C::KEEP ? NB * 4 : 1][MA][4];
        MaxMag mx[MA];
        Terms tq[2];
        if constexpr (C::AHEAD) terms(0, tq[0]);
        auto value = [&](int q, double (&y)[MA][4]) {
            if constexpr (!C::AHEAD) terms(q, tq[q & 1]);
            else if (q + 1 < NB * 4) terms(q + 1, tq[(q + 1) & 1]);
            quad(q, tq[q & 1], y);
        };
#pragma unroll
        for (int q = 0; q < NB * 4; ++q) {
            double(&y)[MA][4] = yk[C::KEEP ? q : 0];
            value(q, y);
#pragma unroll
            for (int a = 0; a < MA; ++a) {
                mx[a].add(y[a][0], y[a][1]);
                mx[a].add(y[a][2], y[a][3]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int a = 0; a < MA; ++a) {
            const int m = swap_reduce<32>(mx[a].word(), Max{});
            if (lane < 32) red[wave * BM + a * 32 + lane] = m;
        }
        __syncthreads();
        double inv[MA];
#pragma unroll
        for (int a = 0; a < MA; ++a) {
            const int r = a * 32 + (lane & 31), m = m0 + r;
            int w = red[r];
#pragma unroll
            for (int i = 1; i < WV; ++i) w = max(w, red[i * BM + r]);
            int ex = max(E_MIN, need_word(w, e.q));
            if (tid < 32 && m < M) {
                ex = clamp_exp_flag(ex, e.flags);
                e.ye[m] = (int8_t)ex;
            }
            inv[a] = pow2(-min(ex, E_MAX));
        }
        if constexpr (!C::KEEP) {
            // nothing of the first pass is kept
#pragma unroll
            for (int a = 0; a < MA; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b) asm volatile("" : "+v"(acc[a][b]));
        }
        if constexpr (!C::KEEP && C::AHEAD) terms(0, tq[0]);
#pragma unroll
        for (int q = 0; q < NB * 4; ++q) {
            double(&y)[MA][4] = yk[C::KEEP ? q : 0];
            if constexpr (!C::KEEP) value(q, y);
#pragma unroll
            for (int a = 0; a < MA; ++a) {
                const uint32_t o = pack4(mant_of(y[a][0], inv[a]), mant_of(y[a][1], inv[a]), mant_of(y[a][2], inv[a]),
                                         mant_of(y[a][3], inv[a]));
                *(uint32_t *)(lds + ort + a * 32 * RP + 8 * q) = o;
            }
            if (!C::KEEP || q & 1) __builtin_amdgcn_sched_barrier(0);
        }
        // y is gone: room for the next tile's loads
        if constexpr (!C::EARLY) fetch_x(next, 0, xn);
        fetch_r(next, rn);
        // the wave's own columns, 16 bytes per lane: its LDS writes come before its
        // reads, and no other wave is waited for
        const bool vec = (N & 15) == 0 && ((uintptr_t)e.y & 15) == 0;
        constexpr int CPW = 2 * NB, LPR = CPW == 6 ? 8 : CPW, RPI = 64 / LPR;  // lanes of a row, rows of a pass
        static_assert(CPW == 4 || CPW == 6 || CPW == 8, "lanes of a row");
        const int frow = (tid & 63) / LPR, fc = wave * 32 * NB + (tid & (LPR - 1)) * 16;
        const bool mine = (tid & (LPR - 1)) < CPW && fc < N;
        int8_t *dst = e.y + (long long)(m0 + frow) * N + fc;
        const int8_t *src = rt + frow * RP + fc;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < BM / RPI; ++i) {
            if (mine && m0 + frow + i * RPI < M) {
                v4i o = *(const v4i *)(src + i * RPI * RP);
                if (e.relu) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = (int)relu4((uint32_t)o[k]);
                }
                int8_t *d = dst + (long long)(i * RPI) * N;
                if (vec) {
                    *(v4i *)d = o;
                } else {
                    const uint32_t v[4] = {(uint32_t)o[0], (uint32_t)o[1], (uint32_t)o[2], (uint32_t)o[3]};
                    store_run<16>(d - fc, fc, N, v);
                }
            }
        }
        if constexpr (RES != RES_NONE) __syncthreads();  // the result is read: room for the next residual
        store_x(xn);
        store_r(rn);
    }
}

hipError_t launch_rows_add(const int8_t *x, const int8_t *w, int M, int N, int K, int8_t *wt, int ni,
                           const AddEpi &e, hipStream_t st) {
    const int ks = rows_steps(K);
    prof_begin(st, PROF_GEMM_ADD);
    hipLaunchKernelGGL(tile_weight_kernel, dim3(8 * ni, (ks + 3) / 4), dim3(256), 0, st, w, N, K, ks, wt);
    auto go = [&](auto ni_tag, auto kc_tag) {
        constexpr int NI = decltype(ni_tag)::value, KC = decltype(kc_tag)::value;
        using C = RowsCfg<NI, KC, RES_NONE>;
        const int tiles = (M + C::BM - 1) / C::BM;
        const dim3 grid(std::min(tiles, C::PER_CU * NCU)), block(C::THR);
        if (!e.r) hipLaunchKernelGGL((rows_add_kernel<NI, KC, RES_NONE>), grid, block, 0, st, x, wt, M, N, K, ks, e);
        else if (e.r_vec) hipLaunchKernelGGL((rows_add_kernel<NI, KC, RES_VEC>), grid, block, 0, st, x, wt, M, N, K, ks, e);
        else hipLaunchKernelGGL((rows_add_kernel<NI, KC, RES_ANY>), grid, block, 0, st, x, wt, M, N, K, ks, e);
    };
#define IE_CASE(NI_, KC_) go(std::integral_constant<int, NI_>{}, std::integral_constant<int, KC_>{})
    // a short contraction takes its steps only
    const bool brief = ks <= 8;
    if (ni == 1 && brief) IE_CASE(1, 8);
    else if (ni == 1) IE_CASE(1, 16);
    else if (ni == 2 && brief) IE_CASE(2, 8);
    else if (ni == 2) IE_CASE(2, 32);
    else if (ni == 3 && brief) IE_CASE(3, 8);
    else if (ni == 3) IE_CASE(3, 32);
    else if (brief) IE_CASE(4, 8);
    else IE_CASE(4, 32);
#undef IE_CASE
    prof_end(st, PROF_GEMM_ADD);
    return hipGetLastError();
}

}  // namespace ie
