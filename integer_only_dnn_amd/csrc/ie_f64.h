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

// Smallest exponent for the magnitude m >= 0 (NEED_NONE when zero): with m in
// [2^x, 2^(x+1)) it is x - q + 1, plus one when the q bits below the leading
// one are all ones (m rounds up to 2^q units).
__device__ __forceinline__ int need_f64(double m, int q) {
    if (m == 0.0) return NEED_NONE;
    const int hi = __double2hiint(m);
    const int ones = (1 << q) - 1;
    return (hi >> 20) - 1023 - q + 1 + ((((hi & 0xfffff) >> (20 - q)) == ones) ? 1 : 0);
}

// The mantissa of v in units of 2^-k (inv = 2^k), half to even, as an int
// whose low byte is the int8.
__device__ __forceinline__ int mant_of(double v, double inv) {
    return __double2loint(__builtin_fma(v, inv, ROUND_MAGIC));
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
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

// A sum or maximum over the T threads of a row (T <= 64: within a wave; more:
// the whole block), in every thread.  `sh` holds one value per wave.
template <int T, class V, class F>
__device__ __forceinline__ V row_reduce(V v, F f, V *sh) {
#pragma unroll
    for (int s = 1; s < (T < 64 ? T : 64); s <<= 1) v = f(v, __shfl_xor(v, s));
    if constexpr (T > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
        __syncthreads();
        v = sh[0];
        for (int i = 1; i < T / 64; ++i) v = f(v, sh[i]);
    }
    return v;
}

struct Add {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
    __device__ __forceinline__ int operator()(int a, int b) const { return max(a, b); }
};

}  // namespace ie
