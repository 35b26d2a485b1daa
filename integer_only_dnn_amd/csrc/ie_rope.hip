// Rotary positions on the rows of (C, e) matrices, and the table of cosines
// and sines they read.
//
// A pair (a, b) of a head's mantissas becomes (a c - b s, a s + b c), c and s
// whole numbers in units of 2^-14; what is not rotated is taken 2^14 times.
// So a row is whole numbers below 2^23 at exponent e - 14 (here below 2^31 in
// units of 2^(e - 22), with their low eight bits zero), exact in fp32, and rounded
// once, at the row's (or the whole tensor's) exponent.  The inverse rotation,
// which is also the gradient, has -s for s.
//
// Bound by the stream over X and Y: 25216 rows of 36 heads of 64 (116 MB) back in
// 24.4 us, 4.8 TB/s of a large copy's 4.9, and 29 from memory (with a branch past what is not rotated,
// which half of every wave's lanes take, 25.9); 16 rows of 48 heads of 128 in 3.3
// us, a launch's time.
#include "ie_f64.h"
#include "ie_internal.h"

#pragma clang fp contract(off)

namespace ie {

constexpr float ROPE_MAGIC = 12582912.0f;  // 1.5 * 2^23

// Row t of the table: (cos, sin) of t f_k for the k-th pair, in 64 bits up to
// the rounding: at position 10^5 a 32-bit angle would be off by 2^-8.
struct RopeFreqs {
    double f[IE_ROPE_MAX / 2];
};
__global__ __launch_bounds__(256) void rope_table_kernel(RopeFreqs fr, int half, long long positions, int *table) {
    const long long n = positions * half;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const long long t = i / half;
        double s, c;
        sincos((double)t * fr.f[i - t * half], &s, &c);
        const int ci = (int)rint(c * 16384.0), si = (int)rint(s * 16384.0);
        table[i] = (ci & 0xffff) | si << 16;
    }
}

// Eight neighbours of a row (or, for the two-halves layout, two runs of four)
// as the numbers they become, in units of 2^(e - 22): two bytes as the upper
// halves of 16-bit numbers, one two-element product of 16-bit integers each.
struct RopeUnit {
    int at[2];  // first column of each run of four
    int k;      // first pair of four, or -1: not rotated
};
__device__ __forceinline__ RopeUnit rope_unit(const RopeArgs &p, int u) {
    const int head = (int)(((uint64_t)(uint32_t)u * p.per.m) >> p.per.s), k = u - head * (p.d >> 3), c0 = head * p.d;
    RopeUnit r;
    const bool on = head < p.heads && 8 * k < p.rot;
    r.k = on ? 4 * k : -1;
    const bool halves = on && !p.interleaved;
    r.at[0] = c0 + (halves ? 4 : 8) * k;
    r.at[1] = halves ? r.at[0] + (p.rot >> 1) : r.at[0] + 4;
    return r;
}
typedef short s2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void rope8(bool interleaved, s2 turn, uint32_t lo, uint32_t hi, const int4 &t, float (&y)[8]) {
    const int w[4] = {t.x, t.y, t.z, t.w};
    uint32_t ab[4];
    if (interleaved) {
        ab[0] = __builtin_amdgcn_perm(lo, lo, 0x010c000cu);
        ab[1] = __builtin_amdgcn_perm(lo, lo, 0x030c020cu);
        ab[2] = __builtin_amdgcn_perm(hi, hi, 0x010c000cu);
        ab[3] = __builtin_amdgcn_perm(hi, hi, 0x030c020cu);
    } else {
        ab[0] = __builtin_amdgcn_perm(hi, lo, 0x040c000cu);
        ab[1] = __builtin_amdgcn_perm(hi, lo, 0x050c010cu);
        ab[2] = __builtin_amdgcn_perm(hi, lo, 0x060c020cu);
        ab[3] = __builtin_amdgcn_perm(hi, lo, 0x070c030cu);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // products with (c, -s) and (s, c), s of the table times turn's first, -s its second
        const s2 cs = __builtin_bit_cast(s2, w[i]), v = __builtin_bit_cast(s2, ab[i]);
        const s2 a = cs * s2{1, turn[1]}, b = s2{cs[1], cs[0]} * s2{turn[0], 1};
        const int ya = __builtin_amdgcn_sdot2(v, a, 0, false), yb = __builtin_amdgcn_sdot2(v, b, 0, false);
        y[interleaved ? 2 * i : i] = (float)ya;
        y[interleaved ? 2 * i + 1 : 4 + i] = (float)yb;
    }
}

__device__ __forceinline__ int rope_position(const RopeArgs &p, long long row, bool tell) {
    const long long t = p.pos ? (long long)p.pos[row] : row;
    if (t >= 0 && t < p.positions) return (int)t;
    if (tell) atomicOr(p.flags, IE_FLAG_INDEX);
    return 0;
}

// T threads per row, NU units each: the smallest T NU that holds the row.  A
// thread's units are the same in every row, so the one division by the head's size
// is done once.
template <int T, int NU, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs p) {
    constexpr int RPB = 256 / T;
    __shared__ int sh[4];
    const int t = threadIdx.x % T, slot = threadIdx.x / T, units = p.cols >> 3;
    const short way = p.inverse ? -1 : 1;
    const s2 turn = {way, (short)-way};
    int run = NEED_NONE;
    int whole = 0;
    RopeUnit un[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) un[i] = rope_unit(p, min(t + T * i, units - 1));
    if (p.mode == NORM_ROUND) {
        int m = NEED_NONE;
        for (int i = threadIdx.x; i < p.n_bmax; i += 256) m = max(m, p.bmax[i]);
        whole = clamp_exp_flag(max(E_MIN, row_reduce<256>(m, Max{}, sh)), p.flags);
        if (blockIdx.x == 0 && threadIdx.x == 0) p.ye[0] = (int8_t)whole;
    }
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += (long long)gridDim.x * RPB) {
        const bool ok = r0 + slot < p.rows;
        const long long row = ok ? r0 + slot : p.rows - 1;
        const int ex = p.xe[p.x_row ? row : 0] - 22;
        const int *tab = p.table + (long long)rope_position(p, row, ok && t == 0 && p.mode != NORM_ROUND) * (p.rot >> 1);
        const int8_t *x = p.x + row * p.cols;
        float y[NU][8];
        uint32_t lo[NU], hi[NU];
        int4 w[NU];
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            lo[i] = *(const uint32_t *)(x + un[i].at[0]);
            hi[i] = *(const uint32_t *)(x + un[i].at[1]);
            w[i] = int4{16384, 16384, 16384, 16384};  // what is not rotated: cos 1, sin 0
            if (un[i].k >= 0) w[i] = *(const int4 *)(tab + un[i].k);
        }
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            rope8(INTER, turn, lo[i], hi[i], w[i], y[i]);  // the last runs of a row may be taken twice
#pragma unroll
            for (int k = 0; k < 8; k += 2) asm("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(big) : "v"(y[i][k]), "v"(y[i][k + 1]));
        }
        int e = whole;
        if (p.mode != NORM_ROUND) {
            const int m = row_reduce<T>((int)big, Max{}, sh);
            const int need = need32(m, ex, p.q);
            if (p.mode == NORM_NEED) {
                run = max(run, need);
                continue;
            }
            e = max(E_MIN, need);
            if (ok && t == 0) {
                e = clamp_exp_flag(e, p.flags);
                p.ye[row] = (int8_t)e;
            }
            e = min(e, E_MAX);
        }
        if (!ok) continue;
        const float inv = __int_as_float((127 + min(max(ex - e, -100), 100)) << 23);
        int8_t *out = p.y + row * p.cols;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            if (t + T * i >= units) continue;
            int o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __float_as_int(__builtin_fmaf(y[i][k], inv, ROPE_MAGIC));
            *(uint32_t *)(out + un[i].at[0]) = pack4(o[0], o[1], o[2], o[3]);
            *(uint32_t *)(out + un[i].at[1]) = pack4(o[4], o[5], o[6], o[7]);
        }
    }
    if (p.mode == NORM_NEED) {
        run = row_reduce<256>(run, Max{}, sh);
        if (threadIdx.x == 0) p.bmax[blockIdx.x] = run;
    }
}

// Element c of a row, for heads whose pairs do not come in runs of four.
__device__ __forceinline__ float rope1(const RopeArgs &p, const int8_t *x, const int *tab, int c, float sign) {
    const int head = c / p.d, j = c - head * p.d, half = p.rot >> 1;
    if (head >= p.heads || j >= p.rot) return 16384.0f * (float)x[c];
    const int k = p.interleaved ? j >> 1 : j < half ? j : j - half;
    const bool second = p.interleaved ? j & 1 : j >= half;
    const int step = p.interleaved ? 1 : half;
    const float co = (float)(int16_t)tab[k], si = sign * (float)(tab[k] >> 16);
    return second ? (float)x[c - step] * si + (float)x[c] * co : (float)x[c] * co - (float)x[c + step] * si;
}

// The same for any head size, alignment and length: a block per row, which it
// walks twice.
__global__ __launch_bounds__(256) void rope_any_kernel(RopeArgs p) {
    __shared__ int sh[4];
    const float sign = p.inverse ? -1.0f : 1.0f;
    int run = NEED_NONE, e = 0;
    if (p.mode == NORM_ROUND) {
        int m = NEED_NONE;
        for (int i = threadIdx.x; i < p.n_bmax; i += 256) m = max(m, p.bmax[i]);
        e = clamp_exp_flag(max(E_MIN, row_reduce<256>(m, Max{}, sh)), p.flags);
        if (blockIdx.x == 0 && threadIdx.x == 0) p.ye[0] = (int8_t)e;
    }
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int ex = p.xe[p.x_row ? row : 0] - 14;
        const int *tab = p.table + (long long)rope_position(p, row, threadIdx.x == 0 && p.mode != NORM_ROUND) * (p.rot >> 1);
        const int8_t *x = p.x + row * p.cols;
        int8_t *out = p.y + row * p.cols;
        if (p.mode != NORM_ROUND) {
            float big = 0.0f;
            for (int c = threadIdx.x; c < p.cols; c += 256) big = fmaxf(big, fabsf(rope1(p, x, tab, c, sign)));
            const int need = need32(row_reduce<256>((int)big, Max{}, sh), ex, p.q);
            if (p.mode == NORM_NEED) {
                run = max(run, need);
                continue;
            }
            e = max(E_MIN, need);
            if (threadIdx.x == 0) {
                e = clamp_exp_flag(e, p.flags);
                p.ye[row] = (int8_t)e;
            }
            e = min(e, E_MAX);
        }
        const float inv = __int_as_float((127 + min(max(ex - e, -100), 100)) << 23);
        for (int c = threadIdx.x; c < p.cols; c += 256)
            out[c] = (int8_t)__float_as_int(__builtin_fmaf(rope1(p, x, tab, c, sign), inv, ROPE_MAGIC));
    }
    if (p.mode == NORM_NEED && threadIdx.x == 0) p.bmax[blockIdx.x] = run;
}

hipError_t launch_rope_table(const double *freqs, int half, long long positions, int16_t *table, hipStream_t st) {
    RopeFreqs f;
    for (int k = 0; k < half; ++k) f.f[k] = freqs[k];
    const long long blocks = (positions * half + 255) / 256;
    prof_begin(st, PROF_ROPE);
    hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, f, half, positions,
                       (int *)table);
    prof_end(st, PROF_ROPE);
    return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs &a, const RopePlan &pl, hipStream_t st) {
    prof_begin(st, PROF_ROPE);
    const dim3 grid((unsigned)pl.grid), block(256);
    bool done = false;
    if (pl.nu == 0) {
        hipLaunchKernelGGL(rope_any_kernel, grid, block, 0, st, a);
        done = true;
    }
#define IE_CASE(T_, N_)                                                               \
    if (pl.t == T_ && pl.nu == N_) {                                                               \
        if (a.interleaved) hipLaunchKernelGGL((rope_kernel<T_, N_, true>), grid, block, 0, st, a); \
        else hipLaunchKernelGGL((rope_kernel<T_, N_, false>), grid, block, 0, st, a);              \
        done = true;                                                                               \
    }
    IE_ROPE_SHAPES(IE_CASE)
#undef IE_CASE
    prof_end(st, PROF_ROPE);
    return done ? hipGetLastError() : hipErrorInvalidValue;
}

}  // namespace ie
