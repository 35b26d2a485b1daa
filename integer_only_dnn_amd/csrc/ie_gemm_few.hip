// Forward product with bias, residual and ReLU for a few rows (single tokens
// and small batches of them, M <= 64): the weight is what has to be read, and
// it is read once, straight into the matrix instructions' registers.
//
// A workgroup takes 16 columns of the result; its 8 waves share out the
// contraction, 64 bytes of 16 weight rows per step and several steps in
// flight, with v_mfma_i32_16x16x64_i8 run transposed (a lane holds one row of
// the result and four neighbouring columns).  X comes from L2.  The waves'
// sums meet in LDS; the workgroup writes them and the largest magnitude of
// each row's 16 results, from which the second kernel has the groups'
// exponents and rounds.
//
// Bound by the two launches and the weight's way from memory: 5 x 4096 x 4096
// takes 9.6 to 10.7 us from box to box, 3.2 of them the weight's 16.8 MB at the
// rate of a large copy (split contractions and the pass that adds them: 23.8).
#include <type_traits>

#include "ie_f64.h"
#include "ie_internal.h"

#pragma clang fp contract(off)

namespace ie {

constexpr int FEW_THR = 512, FEW_WV = FEW_THR / 64, FEW_BN = 16, FEW_ROUND = 256;

// What four neighbours of the result (columns n .. n + 3 of row m) take beside
// their contractions; loaded ahead of them.
struct FewTerms {
    int xe, re, we[4], bm[4], be[4];
    uint32_t r4;
};
__device__ __forceinline__ FewTerms few_terms(const AddEpi &e, int m, int n, int N) {
    FewTerms t;
    t.xe = e.xe[e.x_row ? m : 0];
    t.re = e.r ? e.re[e.r_row ? m : 0] : 0;
    t.r4 = e.r ? load4(e.r + (long long)m * N, n, N) : 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int col = min(n + k, N - 1);
        t.we[k] = e.we[e.w_row ? col : 0];
        t.bm[k] = e.bias.m ? e.bias.m[col] : 0;
        t.be[k] = e.bias.m ? e.bias.e[e.bias.per ? col : 0] : 0;
    }
    return t;
}

// Their values; each fused step is an exact product and one rounded sum.  Past
// N: zero.
__device__ __forceinline__ void few_values(const FewTerms &t, v4i c, int n, int N, double (&y)[4]) {
    const double sx = pow2(t.xe), sr = pow2(t.re);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const double v = __builtin_fma((double)c[k], sx * pow2(t.we[k]), (double)t.bm[k] * pow2(t.be[k]));
        y[k] = n + k < N ? __builtin_fma((double)byte_of(t.r4, k), sr, v) : 0.0;
    }
}

// x [M x K], w [N x K]; acc [M x Np] (Np: N in whole groups
// of 16), word [M][Np / 16], or [Np / 16] for a whole-tensor result.  U: steps in
// flight; EVEN: rows of whole runs of 16 bytes.
template <int MT, int U, bool EVEN>
__global__ __launch_bounds__(FEW_THR) void few_add_kernel(const int8_t *x, const int8_t *w, int M, int N, int K, AddEpi e,
                                                           int *acc, int *word) {
    __shared__ v4i part[FEW_WV][MT * 64];
    __shared__ int shm[MT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n0 = blockIdx.x * FEW_BN;
    const int row = lane & 15, kq = 16 * (lane >> 4);
    const int8_t *wr = w + (long long)min(n0 + row, N - 1) * K;
    const int steps = (K + 63) / 64;
    const int m = wave * 16 + row, n = n0 + 4 * (lane >> 4), nb = gridDim.x;
    FewTerms ft;
    if (wave < MT) ft = few_terms(e, min(m, M - 1), n, N);
    v4i c[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) c[t] = v4i{0, 0, 0, 0};
    for (int s0 = wave; s0 < steps; s0 += FEW_WV * U) {
        v4i a[U], b[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s0 + u * FEW_WV) * 64 + kq;
            if constexpr (EVEN) {
                a[u] = *(const v4i *)(wr + min(k, K - 16));
            } else {
                uint32_t v[4];
                load_run<16>(wr, k, K, v);
                a[u] = v4i{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s0 + u * FEW_WV) * 64 + kq;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int8_t *xr = x + (long long)min(t * 16 + row, M - 1) * K;
                if constexpr (EVEN) {
                    b[u][t] = *(const v4i *)(xr + min(k, K - 16));
                } else {
                    uint32_t v[4];
                    load_run<16>(xr, k, K, v);
                    b[u][t] = v4i{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // past the end of whole runs both factors repeat: X counts as zero
            const bool in = !EVEN || (s0 + u * FEW_WV) * 64 + kq < K;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                v4i v = b[u][t];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = in ? v[i] : 0;
                c[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u], v, c[t], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t * 64 + lane] = c[t];
    __syncthreads();
    if (wave < MT) {
        v4i s = part[0][tid];
#pragma unroll
        for (int i = 1; i < FEW_WV; ++i) s += part[i][tid];
        double y[4];
        MaxMag mx;
        few_values(ft, s, n, N, y);
        mx.add(y[0], y[1]);
        mx.add(y[2], y[3]);
        int g = m < M ? mx.word() : 0;
        g = swap_reduce<32>(swap_reduce<16>(g, Max{}), Max{});
        if (m < M) {
            *(v4i *)(acc + (long long)m * nb * FEW_BN + n) = s;
            if (e.y_row && lane < 16) word[(long long)m * nb + blockIdx.x] = g;
        }
        g = lane_reduce<16>(g, Max{});
        if (lane == 0) shm[wave] = g;
    }
    if (e.y_row) return;
    __syncthreads();
    if (tid == 0) {
        int g = shm[0];
#pragma unroll
        for (int t = 1; t < MT; ++t) g = max(g, shm[t]);
        word[blockIdx.x] = g;
    }
}

// A block rounds FEW_ROUND runs of four columns of a row.
__global__ __launch_bounds__(FEW_ROUND) void few_round_kernel(AddEpi e, const int *acc, const int *word, int M, int N,
                                                              int nb) {
    __shared__ int shi[FEW_ROUND / 64];
    const int m = blockIdx.y, n = (blockIdx.x * FEW_ROUND + threadIdx.x) * 4;
    double y[4];
    if (n < N) few_values(few_terms(e, m, n, N), *(const v4i *)(acc + (long long)m * nb * FEW_BN + n), n, N, y);
    const int *wp = e.y_row ? word + (long long)m * nb : word;
    int g = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < nb; i += FEW_ROUND) g = max(g, wp[i]);
    g = row_reduce<FEW_ROUND>(g, Max{}, shi);
    const int need = max(E_MIN, need_word(g, e.q)), ex = min(need, E_MAX);
    if (blockIdx.x == 0 && threadIdx.x == 0 && (e.y_row || m == 0)) {
        clamp_exp_flag(need, e.flags);
        e.ye[e.y_row ? m : 0] = (int8_t)ex;
    }
    if (n >= N) return;
    const double inv = pow2(-ex);
    uint32_t o = pack4(mant_of(y[0], inv), mant_of(y[1], inv), mant_of(y[2], inv), mant_of(y[3], inv));
    if (e.relu) o = relu4(o);
    store4(e.y + (long long)m * N, n, N, o);
}

hipError_t launch_few_add(const int8_t *x, const int8_t *w, int M, int N, int K, int *acc, int *word,
                          const AddEpi &e, hipStream_t st) {
    const int nb = (N + FEW_BN - 1) / FEW_BN;
    prof_begin(st, PROF_GEMM_ADD);
    auto go = [&](auto mt, auto u) {
        constexpr int MT = decltype(mt)::value, U = decltype(u)::value;
        const dim3 grid(nb), block(FEW_THR);
        if (K % 16 == 0) hipLaunchKernelGGL((few_add_kernel<MT, U, true>), grid, block, 0, st, x, w, M, N, K, e, acc, word);
        else hipLaunchKernelGGL((few_add_kernel<MT, U, false>), grid, block, 0, st, x, w, M, N, K, e, acc, word);
    };
#define IE_CASE(MT_, U_) go(std::integral_constant<int, MT_>{}, std::integral_constant<int, U_>{})
    const bool brief = K <= 2 * 64 * FEW_WV;  // two steps a wave
    if (M <= 16 && brief) IE_CASE(1, 2);
    else if (M <= 16) IE_CASE(1, 8);
    else if (M <= 32 && brief) IE_CASE(2, 2);
    else if (M <= 32) IE_CASE(2, 8);
    else if (brief) IE_CASE(4, 2);
    else IE_CASE(4, 4);
#undef IE_CASE
    prof_end(st, PROF_GEMM_ADD);
    prof_begin(st, PROF_SPLIT_ADD);
    hipLaunchKernelGGL(few_round_kernel, dim3((N + 4 * FEW_ROUND - 1) / (4 * FEW_ROUND), M), dim3(FEW_ROUND), 0, st, e,
                       acc, word, M, N, nb);
    prof_end(st, PROF_SPLIT_ADD);
    return hipGetLastError();
}

}  // namespace ie
