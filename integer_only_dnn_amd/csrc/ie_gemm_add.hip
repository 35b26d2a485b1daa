// Forward product with bias, residual and ReLU in its epilogue:
//   y = (acc 2^(e_X + e_W) + bias) + R,
// acc the exact int32 contraction, each sum rounded to 53 bits (exact while
// its terms span no more), y rounded once into Y's groups, then the clip on
// the rounded mantissas.
//
// The contraction is the dense products' (gemm_tile); its matrix
// instructions run transposed, so that a lane holds one row of the result
// and four neighbouring columns per accumulator quarter: a row's maximum is
// taken in registers, the residual is read and the result written four bytes
// at a time, and the bias is the same for the 32 lanes of a half-wave.  The
// two products of an element (by the scales' powers of two) are exact in the
// fp64 unit, which runs its fused multiply-add at the fp32 rate.
//
// Whole-tensor results, and rows that do not lie whole in a workgroup, leave
// rounded to odd as int16 and take a second pass: 25216 x 768 x 768 with a
// residual into a whole-tensor result 43 + 11 us, bound by the epilogue's fp64
// instructions, the int16 values' way through memory and back next.
#include "ie_f64.h"
#include "ie_gemm_impl.h"

namespace ie {

template <bool RES>
struct EpiAdd {
    AddEpi e;

    // a tile of int8 or int16 results from LDS to memory, 16 bytes per thread;
    // int16 rows are add_pitch(N) apart, zeros past N
    template <int ES, int BM, int BN>
    __device__ __forceinline__ void flush(const int8_t *lds, void *dst, int m0, int n0, int M, int n, bool vec) const {
        constexpr int PITCH = BN * ES + 16, CPR = BN * ES / 16, EPC = 16 / ES;
        const int N = ES == 2 ? add_pitch(n) : n;
#pragma unroll
        for (int q0 = 0; q0 < BM * CPR; q0 += NTHR) {
            const int q = q0 + threadIdx.x, row = q / CPR, cb = q % CPR * 16;
            const int gr = m0 + row, gc = n0 + cb / ES;
            if (gr >= M || gc >= N) continue;
            v4i v = *(const v4i *)(lds + row * PITCH + cb);
            if (ES == 1 && e.relu) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = (int)relu4((uint32_t)v[k]);
            }
            int8_t *g = (int8_t *)dst + ((long long)gr * N + gc) * ES;
            if (ES == 2 || (vec && gc + EPC <= N)) {
                *(v4i *)g = v;
            } else {
                const int bytes = min(16, (N - gc) * ES);
#pragma unroll
                for (int k = 0; k < 4; ++k) store4(g, 4 * k, bytes, (uint32_t)v[k]);
            }
        }
    }

    template <int MI, int NI, int RG, int DI, int AM, int AN>
    __device__ __forceinline__ void finish(const v16i (&acc)[AM][AN], int8_t *lds, int m0, int n0, int tile_m,
                                           int tile_n, int M, int N, int TM) const {
        constexpr int BM = 64 * MI, BN = 64 * NI, RP = BN + 4;  // RP: pitch of the residual tile
        int tid = threadIdx.x;
        // offsets made of the thread's number are made here: kept over the contraction,
        // they would not fit the registers
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
        double *cs = (double *)lds, *bs = cs + BN;  // column scales, bias
        int *red = (int *)(bs + BN);               // maxima [2][BM]
        int8_t *rt = (int8_t *)(red + 2 * BM), *out = rt + BM * RP;
        static_assert(16 * BN + 8 * BM + BM * RP + BM * (BN * 2 + 16) <= TileLds<LD_K, LD_K, MI, NI, false>::value,
                      "epilogue exceeds the tile's LDS");
        static_assert(BM * RP % 16 == 0, "staging alignment");
        __syncthreads();  // every wave is done with the last stage
        for (int i = tid; i < BN; i += NTHR) {
            const int n = n0 + i;
            // past the last column everything is zero
            cs[i] = n < N ? pow2((int)e.we[e.w_row ? n : 0]) : 0.0;
            bs[i] = n < N && e.bias.m ? (double)e.bias.m[n] * pow2((int)e.bias.e[e.bias.per ? n : 0]) : 0.0;
        }
        if constexpr (RES) {
            constexpr int CPR = BN / 16;
#pragma unroll
            for (int q0 = 0; q0 < BM * CPR; q0 += NTHR) {
                const int q = q0 + tid, row = q / CPR, c = q % CPR * 16;
                uint32_t v[4] = {0, 0, 0, 0};
                if (m0 + row < M && n0 + c < N) {
                    const int8_t *src = e.r + (long long)(m0 + row) * N + n0;
                    if (e.r_vec) {
                        const v4i w = *(const v4i *)(src + c);
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = (uint32_t)w[k];
                    } else {
                        const int8_t *rowp = src - n0;
                        if (N >= 16) {
                            const v4i w = load16(rowp, n0 + c, N);
#pragma unroll
                            for (int k = 0; k < 4; ++k) v[k] = (uint32_t)w[k];
                        } else {
                            load_run<16>(rowp, n0 + c, N, v);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) *(uint32_t *)(rt + row * RP + c + 4 * k) = v[k];
            }
        }
        __syncthreads();

        double y[MI][NI][16], sx[MI], sr[MI];
        MaxMag mx[MI];
        int row[MI];
#pragma unroll
        for (int a = 0; a < MI; ++a) {
            row[a] = wm * 32 * MI + a * 32 + (lane & 31);
            const int m = m0 + row[a];
            sx[a] = m < M ? pow2((int)e.xe[e.x_row ? m : 0]) : 0.0;
            sr[a] = RES && m < M ? pow2((int)e.re[e.r_row ? m : 0]) : 0.0;
        }
#pragma unroll
        for (int b = 0; b < NI; ++b)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int c = wn * 32 * NI + b * 32 + 8 * h + 4 * (lane >> 5);
#pragma unroll
                for (int a = 0; a < MI; ++a) {
                    const uint32_t r4 = RES ? *(const uint32_t *)(rt + row[a] * RP + c) : 0u;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // each fused step is an exact product and one rounded sum
                        double v = __builtin_fma((double)acc[a][b][4 * h + k], sx[a] * cs[c + k], bs[c + k]);
                        if constexpr (RES) v = __builtin_fma((double)byte_of(r4, k), sr[a], v);
                        y[a][b][4 * h + k] = v;
                        if (k % 2) mx[a].add(y[a][b][4 * h + k - 1], v);
                    }
                }
                if (h & 1) __builtin_amdgcn_sched_barrier(0);
            }
        // the group's exponent (results in this pass), or the round-to-odd
        // position two bits below the tile's own need
        double inv[MI];
        if constexpr (RG) {
#pragma unroll
            for (int a = 0; a < MI; ++a) {
                const int m = swap_reduce<32>(mx[a].word(), Max{});
                if (lane < 32) red[wn * BM + row[a]] = m;
            }
            __syncthreads();
#pragma unroll
            for (int a = 0; a < MI; ++a) {
                const int need = need_word(max(red[row[a]], red[BM + row[a]]), e.q), m = m0 + row[a];
                const bool first = lane < 32 && wn == 0 && m < M;
                if constexpr (DI) {
                    int ex = max(E_MIN, need);
                    if (first) {
                        ex = clamp_exp_flag(ex, e.flags);
                        e.ye[m] = (int8_t)ex;
                    }
                    inv[a] = pow2(-min(ex, E_MAX));
                } else {
                    if (first) e.p16[(long long)m * ((N + BN - 1) / BN) + tile_n] = (int16_t)(need == NEED_NONE ? P_NONE : need);
                    inv[a] = need == NEED_NONE ? 0.0 : pow2(2 - need);
                }
            }
        } else {
            int t = 0;
#pragma unroll
            for (int a = 0; a < MI; ++a) t = max(t, m0 + row[a] < M ? mx[a].word() : 0);
            t = lane_reduce<64>(t, Max{});
            if (lane == 0) red[wave] = t;
            __syncthreads();
            const int need = need_word(max(max(red[0], red[1]), max(red[2], red[3])), e.q);
            double in;
            if constexpr (DI) {
                const int ex = clamp_exp_flag(max(E_MIN, need), e.flags);
                if (tid == 0) e.ye[0] = (int8_t)ex;
                in = pow2(-ex);
            } else {
                if (tid == 0) e.p16[tile_m + TM * tile_n] = (int16_t)(need == NEED_NONE ? P_NONE : need);
                in = need == NEED_NONE ? 0.0 : pow2(2 - need);
            }
#pragma unroll
            for (int a = 0; a < MI; ++a) inv[a] = in;
        }
#pragma unroll
        for (int a = 0; a < MI; ++a)
#pragma unroll
            for (int b = 0; b < NI; ++b)
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int c = wn * 32 * NI + b * 32 + 8 * h + 4 * (lane >> 5);
                    const double *v = &y[a][b][4 * h];
                    if constexpr (DI) {
                        *(uint32_t *)(out + row[a] * (BN + 16) + c) =
                            pack4(mant_of(v[0], inv[a]), mant_of(v[1], inv[a]), mant_of(v[2], inv[a]),
                                  mant_of(v[3], inv[a]));
                    } else {
                        // floor, with the lowest bit set where anything is cut off
                        int o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const double w = v[k] * inv[a], f = __builtin_floor(w);
                            o[k] = (int)f | (int)(w != f);
                        }
                        v2i p = {(o[0] & 0xffff) | o[1] << 16, (o[2] & 0xffff) | o[3] << 16};
                        *(v2i *)(out + row[a] * (2 * BN + 16) + 2 * c) = p;
                    }
                    if (h & 1) __builtin_amdgcn_sched_barrier(0);
                }
        __syncthreads();
        if constexpr (DI) flush<1, BM, BN>(out, e.y, m0, n0, M, N, (N & 15) == 0 && ((uintptr_t)e.y & 15) == 0);
        else flush<2, BM, BN>(out, e.v16, m0, n0, M, N, true);
    }
};

template <int MI, int NI, int RG, int DI, bool RES>
__global__ __launch_bounds__(NTHR, (NI == 4 ? 1 : Occ<MI, NI>::value)) void gemm_add_kernel(Operand A, Operand B, int M, int N, int K,
                                                                              int TM, EpiAdd<RES> ep) {
    __shared__ __attribute__((aligned(16))) int8_t lds[TileLds<LD_K, LD_K, MI, NI, false>::value];
    gemm_tile<LD_K, LD_K, MI, NI, false, false, -1, RG, DI>(A, B, M, N, K, K, TM, 1, ep, blockIdx.x, gridDim.x, lds);
}

template <int MI, int NI, bool RES>
static void launch_tile(const Operand &A, const Operand &B, int M, int N, int K, bool direct, const AddEpi &e,
                        hipStream_t st) {
    const int TM = (M + 64 * MI - 1) / (64 * MI), TN = (N + 64 * NI - 1) / (64 * NI);
    const dim3 grid(TM * TN), block(NTHR);
    const EpiAdd<RES> ep{e};
    if (e.y_row) {
        if (direct) hipLaunchKernelGGL((gemm_add_kernel<MI, NI, 1, 1, RES>), grid, block, 0, st, A, B, M, N, K, TM, ep);
        else hipLaunchKernelGGL((gemm_add_kernel<MI, NI, 1, 0, RES>), grid, block, 0, st, A, B, M, N, K, TM, ep);
    } else {
        if (direct) hipLaunchKernelGGL((gemm_add_kernel<MI, NI, 0, 1, RES>), grid, block, 0, st, A, B, M, N, K, TM, ep);
        else hipLaunchKernelGGL((gemm_add_kernel<MI, NI, 0, 0, RES>), grid, block, 0, st, A, B, M, N, K, TM, ep);
    }
}

hipError_t launch_gemm_add(const Operand &A, const Operand &B, int M, int N, int K, Tile t, bool direct,
                           const AddEpi &e, hipStream_t st) {
    prof_begin(st, PROF_GEMM_ADD);
#define IE_CASE(a, b) \
    if (t.mi == a && t.ni == b) {                                              \
        if (e.r) launch_tile<a, b, true>(A, B, M, N, K, direct, e, st);        \
        else launch_tile<a, b, false>(A, B, M, N, K, direct, e, st);           \
    }
    IE_TILES_ADD(IE_CASE)
#undef IE_CASE
    prof_end(st, PROF_GEMM_ADD);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Round-to-odd results (units of 2^(need - 2), the need of their row in the
// tile or of the tile) rounded at their group's largest need.  A value has at
// most 11 bits, so one fp32 fused multiply-add on it rounds half to even into
// the low bits of the sum.  T lanes per row, runs of eight values, CH of them
// in flight: a stream of three bytes a value, 25216 x 768 11 us (7.6 at the rate
// of a large copy).
// ---------------------------------------------------------------------------

template <int T, int CH>
__global__ __launch_bounds__(256) void add_round_kernel(AddEpi e, int M, int N, int lbm, int lbn, int TM, int TN) {
    constexpr int RPB = 256 / T;
    __shared__ int shi[4];
    const int t = threadIdx.x % T, slot = threadIdx.x / T;
    int ex = E_MIN;
    if (!e.y_row) {
        int m = NEED_NONE;
        const long long n = (long long)TM * TN;
        for (long long i = threadIdx.x; i < n; i += 256) m = max(m, (int)e.p16[i]);
        m = row_reduce<256>(m, Max{}, shi);
        ex = clamp_exp_flag(max(E_MIN, m), e.flags);
        if (blockIdx.x == 0 && threadIdx.x == 0) e.ye[0] = (int8_t)ex;
    }
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < M; r0 += (long long)gridDim.x * RPB) {
        const long long row = min(r0 + slot, (long long)M - 1);
        const int16_t *v = e.v16 + row * add_pitch(N), *p = e.y_row ? e.p16 + row * TN : e.p16 + (row >> lbm);
        if (e.y_row) {
            int m = NEED_NONE;
            for (int j = t; j < TN; j += T) m = max(m, (int)p[j]);
            ex = max(E_MIN, lane_reduce<T>(m, Max{}));
            if (t == 0 && r0 + slot < M) {
                ex = clamp_exp_flag(ex, e.flags);
                e.ye[row] = (int8_t)ex;
            }
            ex = min(ex, E_MAX);
        }
        if (r0 + slot >= M) continue;
        for (int c0 = 8 * t; c0 < N; c0 += 8 * T * CH) {
            v4i w[CH];
            int need[CH];
#pragma unroll
            for (int h = 0; h < CH; ++h) {
                const int c = c0 + 8 * T * h < N ? c0 + 8 * T * h : c0;  // past the end: read again, not stored
                w[h] = *(const v4i *)(v + c);
                need[h] = p[(long long)(c >> lbn) * (e.y_row ? 1 : TM)];
            }
#pragma unroll
            for (int h = 0; h < CH; ++h) {
                // P_NONE: all zeros, whatever the shift
                const float s = __builtin_ldexpf(1.0f, max(need[h] - 2 - ex, -100));
                uint32_t o[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    int b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int x = i & 1 ? w[h][2 * k + i / 2] >> 16 : (int)(int16_t)w[h][2 * k + i / 2];
                        b[i] = __float_as_int(__builtin_fmaf((float)x, s, 12582912.0f));  // 1.5 * 2^23
                    }
                    o[k] = pack4(b[0], b[1], b[2], b[3]);
                    if (e.relu) o[k] = relu4(o[k]);
                }
                store_run<8>(e.y + row * N, c0 + 8 * T * h, N, o);
            }
        }
    }
}

hipError_t launch_add_round(const AddEpi &e, int M, int N, Tile t, hipStream_t st) {
    auto lg = [](int v) { int l = 0; while ((1 << l) < v) ++l; return l; };  // tile sides are powers of two
    const int lbm = lg(t.bm()), lbn = lg(t.bn()), TM = (M + t.bm() - 1) / t.bm(), TN = (N + t.bn() - 1) / t.bn();
    auto grid = [&](int rpb) { const int g = (M + rpb - 1) / rpb; return dim3(g < 8 * NCU ? g : 8 * NCU); };
    prof_begin(st, PROF_RTO_FINALIZE);
#define IE_CASE(T_, CH_) \
    hipLaunchKernelGGL((add_round_kernel<T_, CH_>), grid(256 / T_), dim3(256), 0, st, e, M, N, lbm, lbn, TM, TN)
    if (N <= 64) IE_CASE(8, 1);
    else if (N <= 256) IE_CASE(32, 1);
    else if (N <= 512) IE_CASE(32, 2);
    else if (N <= 768) IE_CASE(32, 3);
    else if (N <= 1024) IE_CASE(32, 4);
    else IE_CASE(64, 4);
#undef IE_CASE
    prof_end(st, PROF_RTO_FINALIZE);
    return hipGetLastError();
}

// Both operands' rows to whole runs of 16 bytes, one run per thread.
__global__ __launch_bounds__(256) void pad_two_kernel(const int8_t *x, long long nx, const int8_t *w, long long nw, int K,
                                                      int runs, int8_t *xp, int8_t *wp) {
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < nx + nw; i += gridDim.x * 256ll) {
        const bool first = i < nx;
        const long long j = first ? i : i - nx, row = j / runs;
        uint32_t v[4];
        load_run<16>((first ? x : w) + row * K, (int)(j - row * runs) * 16, K, v);
        *(v4i *)((first ? xp : wp) + j * 16) = v4i{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
    }
}

hipError_t launch_pad_two(const int8_t *x, int M, const int8_t *w, int N, int K, int Kp, int8_t *xp, int8_t *wp,
                          hipStream_t st) {
    const int runs = Kp / 16;
    const long long nx = (long long)M * runs, nw = (long long)N * runs, g = (nx + nw + 255) / 256;
    hipLaunchKernelGGL(pad_two_kernel, dim3(g < 8 * NCU ? (int)g : 8 * NCU), dim3(256), 0, st, x, nx, w, nw, K, runs, xp,
                       wp);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Split contractions: the int32 partials of `splits` chunks summed (|sum| <
// 2^30), then the same epilogue, one block per row at a time.
// ---------------------------------------------------------------------------

__device__ __forceinline__ double split_value(const AddEpi &e, const int *p, int splits, long long stride, long long m,
                                              int n, int N, double sx, double sr) {
    int s = 0;
    const long long o = m * N + n;
    for (int i = 0; i < splits; ++i) s += p[i * stride + o];
    const double bias = e.bias.m ? (double)e.bias.m[n] * pow2((int)e.bias.e[e.bias.per ? n : 0]) : 0.0;
    double v = __builtin_fma((double)s, sx * pow2((int)e.we[e.w_row ? n : 0]), bias);
    if (e.r) v = __builtin_fma((double)e.r[o], sr, v);
    return v;
}

__global__ __launch_bounds__(1024) void split_add_kernel(AddEpi e, const int *partial, int splits, long long stride,
                                                         int M, int N, int mode, int *bmax, int n_bmax) {
    __shared__ int shi[16];
    double inv = 0.0;
    int run = 0;
    if (mode == NORM_ROUND) {
        int m = NEED_NONE;
        for (int i = threadIdx.x; i < n_bmax; i += 1024) m = max(m, bmax[i]);
        m = row_reduce<1024>(m, Max{}, shi);
        const int ex = clamp_exp_flag(max(E_MIN, m), e.flags);
        inv = pow2(-ex);
        if (blockIdx.x == 0 && threadIdx.x == 0) e.ye[0] = (int8_t)ex;
    }
    for (int m = blockIdx.x; m < M; m += gridDim.x) {
        const double sx = pow2((int)e.xe[e.x_row ? m : 0]), sr = e.r ? pow2((int)e.re[e.r_row ? m : 0]) : 0.0;
        if (mode != NORM_ROUND) {
            MaxMag mx;
            for (long long n = threadIdx.x; n < N; n += 1024)
                mx.add(split_value(e, partial, splits, stride, m, (int)n, N, sx, sr), 0.0);
            if (mode == NORM_NEED) {
                run = max(run, mx.word());
                continue;
            }
            int ex = max(E_MIN, need_word(row_reduce<1024>(mx.word(), Max{}, shi), e.q));
            if (threadIdx.x == 0) {
                ex = clamp_exp_flag(ex, e.flags);
                e.ye[m] = (int8_t)ex;
            }
            inv = pow2(-min(ex, E_MAX));
        }
        for (long long n = threadIdx.x; n < N; n += 1024) {
            const int c = (int8_t)mant_of(split_value(e, partial, splits, stride, m, (int)n, N, sx, sr), inv);
            e.y[(long long)m * N + n] = (int8_t)(e.relu && c < 0 ? 0 : c);
        }
    }
    if (mode == NORM_NEED) {
        run = row_reduce<1024>(run, Max{}, shi);
        if (threadIdx.x == 0) bmax[blockIdx.x] = need_word(run, e.q);
    }
}

hipError_t launch_split_add(const AddEpi &e, const int *partial, int splits, int M, int N, int *bmax, hipStream_t st) {
    const int grid = M < SPLIT_ADD_BLOCKS ? M : SPLIT_ADD_BLOCKS;
    const long long stride = (long long)M * N;
    prof_begin(st, PROF_SPLIT_ADD);
    if (e.y_row) {
        hipLaunchKernelGGL(split_add_kernel, dim3(grid), dim3(1024), 0, st, e, partial, splits, stride, M, N, NORM_ROWS,
                           bmax, 0);
    } else {
        hipLaunchKernelGGL(split_add_kernel, dim3(grid), dim3(1024), 0, st, e, partial, splits, stride, M, N, NORM_NEED,
                           bmax, grid);
        hipLaunchKernelGGL(split_add_kernel, dim3(grid), dim3(1024), 0, st, e, partial, splits, stride, M, N, NORM_ROUND,
                           bmax, grid);
    }
    prof_end(st, PROF_SPLIT_ADD);
    return hipGetLastError();
}

}  // namespace ie
