// (C, e) values in the fp64 unit: exact powers of two, the smallest exponent
// of a magnitude, rounding into mantissas, and rows of int8 mantissas handled
// four at a time.  Files that include this allow no contraction, so that
// every written operation rounds by itself.
#pragma once

#include "ie_device.h"

#pragma clang fp contract(off)

namespace ie {

// 2^e, -1022 <= e <= 1023.
__device__ __forceinline__ double pow2(int e) { return __hiloint2double((e + 1023) << 20, 0); }

// 1.5 * 2^52: added to |v| <= 2^51 it leaves v rounded half to even in the
// low bits of the sum.
constexpr double ROUND_MAGIC = 6755399441055744.0;

__device__ __forceinline__ double rint_magic(double v) { return (v + ROUND_MAGIC) - ROUND_MAGIC; }

// The mantissa of v in units of 2^-k (inv = 2^k), half to even, as an int
// whose low byte is the int8.
__device__ __forceinline__ int mant_of(double v, double inv) {
    return __double2loint(__builtin_fma(v, inv, ROUND_MAGIC));
}

// N C - S of byte k of w ^ 0x80808080 (C + 128), s128 = S + 128 N: exact, every
// term below 2^23, and the byte is taken by the conversion itself.
__device__ __forceinline__ double centred(uint32_t w, int k, float n, float s128) {
    return (double)__builtin_fmaf((float)(w >> (8 * k) & 255u), n, -s128);
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    const uint32_t lo = __builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm((uint32_t)d, (uint32_t)c, 0x0c0c0400u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// Four neighbours of a row from column c (any alignment); past n: zeros.
__device__ __forceinline__ uint32_t load4(const int8_t *row, int c, int n) {
    uint32_t w = 0;
    if (c + 4 <= n) {
        __builtin_memcpy(&w, row + c, 4);
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (c + k < n) w |= (uint32_t)(uint8_t)row[c + k] << (8 * k);
    }
    return w;
}

__device__ __forceinline__ void store4(int8_t *row, int c, int n, uint32_t w) {
    if (c + 4 <= n) {
        __builtin_memcpy(row + c, &w, 4);
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (c + k < n) row[c + k] = (int8_t)(w >> (8 * k));
    }
}

__device__ __forceinline__ int byte_of(uint32_t w, int k) { return (int)(int8_t)(w >> (8 * k)); }

struct Add {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ int operator()(int a, int b) const { return max(a, b); }
};

template <int CTRL>
__device__ __forceinline__ int dpp_of(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, true); }
template <int CTRL>
__device__ __forceinline__ double dpp_of(double v) {
    return __hiloint2double(dpp_of<CTRL>(__double2hiint(v)), dpp_of<CTRL>(__double2loint(v)));
}

// f over a lane and its partner 16 (or 32) lanes away: swapping the odd rows
// of one copy with the even rows of another leaves both partners' values.
template <int D, class F>
__device__ __forceinline__ int swap_reduce(int v, F f) {
    const auto r = D == 16 ? __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false)
                           : __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
    return f((int)r[0], (int)r[1]);
}
template <int D, class F>
__device__ __forceinline__ double swap_reduce(double v, F f) {
    const uint32_t h = (uint32_t)__double2hiint(v), l = (uint32_t)__double2loint(v);
    const auto a = D == 16 ? __builtin_amdgcn_permlane16_swap(h, h, false, false)
                           : __builtin_amdgcn_permlane32_swap(h, h, false, false);
    const auto b = D == 16 ? __builtin_amdgcn_permlane16_swap(l, l, false, false)
                           : __builtin_amdgcn_permlane32_swap(l, l, false, false);
    return f(__hiloint2double((int)a[0], (int)b[0]), __hiloint2double((int)a[1], (int)b[1]));
}

// A sum or maximum over groups of T <= 64 lanes, in every lane of the group
// (all lanes active): neighbours, pairs, the mirrored half row, the mirrored
// row, then rows.  Data-parallel moves and swaps, no trip through LDS.
template <int T, class V, class F>
__device__ __forceinline__ V lane_reduce(V v, F f) {
    if constexpr (T >= 2) v = f(v, dpp_of<0xB1>(v));    // lanes 1 0 3 2
    if constexpr (T >= 4) v = f(v, dpp_of<0x4E>(v));    // lanes 2 3 0 1
    if constexpr (T >= 8) v = f(v, dpp_of<0x141>(v));   // half row mirrored
    if constexpr (T >= 16) v = f(v, dpp_of<0x140>(v));  // row mirrored
    if constexpr (T >= 32) v = swap_reduce<16>(v, f);
    if constexpr (T >= 64) v = swap_reduce<32>(v, f);
    return v;
}

// The same over T threads: within a wave, or over a whole block of T; `sh`
// holds a value per wave.
template <int T, class V, class F>
__device__ __forceinline__ V row_reduce(V v, F f, V *sh) {
    v = lane_reduce<(T < 64 ? T : 64)>(v, f);
    if constexpr (T > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
        __syncthreads();
        v = sh[0];
#pragma unroll
        for (int i = 1; i < T / 64; ++i) v = f(v, sh[i]);
    }
    return v;
}

// The same with one barrier: `sh` is not written again before the block has
// met at another one.
template <int T, class V, class F>
__device__ __forceinline__ V row_reduce_once(V v, F f, V *sh) {
    v = lane_reduce<(T < 64 ? T : 64)>(v, f);
    if constexpr (T > 64) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
        __syncthreads();
        v = sh[0];
#pragma unroll
        for (int i = 1; i < T / 64; ++i) v = f(v, sh[i]);
    }
    return v;
}

// Largest magnitude of a run of values, as the high word of its double (the
// need of a magnitude takes its exponent and leading bits only).  High words
// of magnitudes order like the floats of the same bits, so one three-operand
// fp32 maximum, its operands' signs dropped, takes two values; no double
// here reaches the 2^1017 whose high word would be a NaN, or the 2^-1015
// whose high word would be a denormal.
struct MaxMag {
    float m = 0.0f;
    __device__ __forceinline__ void add(double a, double b) {
        const int ha = __double2hiint(a), hb = __double2hiint(b);
        asm("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(m) : "v"(ha), "v"(hb));
    }
    __device__ __forceinline__ int word() const { return __float_as_int(m); }
};

// Smallest exponent for the magnitude whose high word is w (NEED_NONE when
// zero): with m in [2^x, 2^(x+1)) it is x - q + 1, plus one when the q bits
// below the leading one are all ones (m rounds up to 2^q units).
__device__ __forceinline__ int need_word(int w, int q) {
    if (w == 0) return NEED_NONE;
    const int ones = (1 << q) - 1;
    return (w >> 20) - 1023 - q + 1 + ((((w & 0xfffff) >> (20 - q)) == ones) ? 1 : 0);
}

// A run of CH = 4, 8 or 16 mantissas of a row from column c, four to a word;
// past n: zeros.
template <int CH>
__device__ __forceinline__ void load_run(const int8_t *row, int c, int n, uint32_t *w) {
#pragma unroll
    for (int k = 0; k < CH / 4; ++k) w[k] = 0;
    if (c + CH <= n) {
        __builtin_memcpy(w, row + c, CH);
    } else if (c < n) {
#pragma unroll
        for (int k = 0; k < CH / 4; ++k) w[k] = load4(row, c + 4 * k, n);
    }
}

// Bytes c .. c + 15 of a row of n >= 16 (c < n, any alignment; past n: zeros) in
// one load: at the row's end its last 16 bytes, moved down.
__device__ __forceinline__ v4i load16(const int8_t *row, int c, int n) {
    uint64_t v[2];
    __builtin_memcpy(v, row + min(c, n - 16), 16);
    if (c > n - 16) {
        const int s = 8 * (c - (n - 16));
        v[0] = s < 64 ? v[0] >> s | v[1] << (64 - s) : v[1] >> (s - 64);
        v[1] = s < 64 ? v[1] >> s : 0;
    }
    return v4i{(int)v[0], (int)(v[0] >> 32), (int)v[1], (int)(v[1] >> 32)};
}

template <int CH>
__device__ __forceinline__ void store_run(int8_t *row, int c, int n, const uint32_t *w) {
    if (c + CH <= n) {
        __builtin_memcpy(row + c, w, CH);
    } else if (c < n) {
#pragma unroll
        for (int k = 0; k < CH / 4; ++k) store4(row, c + 4 * k, n, w[k]);
    }
}

// The columns of a row that a thread holds when T threads share it, E each:
// runs of CH neighbours (as wide as one load can be), run i of thread t from
// column CH (i T + t).  Rows are read whole runs at a time: a run that crosses
// the row's end takes in the next row's first bytes, one past it the row's
// first ones, and `mask` clears both; only at the matrix's last rows, where
// nothing may follow, is such a run read byte by byte.
template <int T, int E>
struct Cols {
    static constexpr int CH = E % 16 == 0 ? 16 : E % 8 == 0 ? 8 : 4, NC = E / CH, W = E / 4;
    int t, n;
    bool exact;  // every run of every thread lies inside the row
    int at[NC];
    uint32_t mask[W];
    static __device__ __forceinline__ int col(int j, int t) { return CH * (j / CH * T + t) + j % CH; }
    __device__ __forceinline__ int col(int j) const { return col(j, t); }
    __device__ __forceinline__ void init(int t_, int n_) {
        t = t_;
        n = n_;
        exact = n == T * E;
#pragma unroll
        for (int i = 0; i < NC; ++i) at[i] = CH * (i * T + t) < n ? CH * (i * T + t) : 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int left = n - col(4 * i);
            mask[i] = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        }
    }
    // `whole`: a run may be read past the row's end (CH more rows follow, or
    // no run crosses it)
    __device__ __forceinline__ void load(const int8_t *row, bool whole, uint32_t (&w)[W]) const {
        if (whole) {
#pragma unroll
            for (int i = 0; i < NC; ++i) __builtin_memcpy(w + i * CH / 4, row + at[i], CH);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = col(4 * i) < n ? load4(row, col(4 * i), n) : 0u;
        }
    }
    __device__ __forceinline__ void clear(uint32_t (&w)[W]) const {
        if (exact) return;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] &= mask[i];
    }
    __device__ __forceinline__ void store(int8_t *row, const uint32_t (&w)[W]) const {
#pragma unroll
        for (int i = 0; i < NC; ++i) store_run<CH>(row, CH * (i * T + t), n, w + i * CH / 4);
    }
};

}  // namespace ie
