// What the attention kernels share: softmax weights, their digits, tiles of
// heads in LDS and the sequences of a packed batch.
//
// A weight.  A row's scores are t_j = (q . k_j) 2^(e_j), exact in fp32 (at
// most 21 bits), and its largest one is m.  With d = t_j - m rounded to fp32
// and r = scale log2(e) 2^(e_i), the exponent of the weight is d r at a
// resolution of 2^-17, from -32 to 0:
//   y = rint(d r 2^17) 2^-17,  w = 32512 2^floor(y) P(y - floor(y)),
// P(f) = 2^f to 1.1e-4, of degree three, P(0) = 1, P(1) = 2.  Adding 96 to d r
// in one fused multiply-add leaves y in the low bits of a float in [64, 96],
// whose bits 17..22 are floor(y) + 32 and whose fraction is y's: ten
// instructions a weight from the int32 product on, the exponential itself
// eight.  The unit resolution of 2^-17 and the polynomial's error are an
// order below half a step of the 7-bit mantissas that come out.
//
// Digits.  A weight enters a product as an integer n = rint(w ...) of at most
// 32512, as two signed digits n = 256 a + b, a and b int8, so that its sums
// are exact int32 sums of v_mfma_i32_16x16x64_i8 and the order of keys, of
// tiles and of workgroups is of no account.  n + 128 comes out of the adder of
// rint (a magic constant), its two low bytes are a and b + 128.
//
// Fine weights.  Where many weights of a row are small beside its largest, as in
// a long row with one key far ahead of the others, R(w) takes too much of them:
// every weight below half a unit counts as nothing.  Up to ATT_CHECK keys that is
// less than 32512 / 32 in all.  A row that sees more has its sum L taken in units
// of 2^-7 beside it (whole numbers, exact modulo 2^32).  Where the two differ by
// more than a 32nd, or where the head's largest sum of values is below 64 a key, half a
// unit times 128, so that rounding may reach it, all weights of the row are
// taken again with ATT_FINE bits behind their unit, in four digits (the sums
// of 131071 keys stay below 2^53).  The mark of such a row is the last bit of its
// maximum (scores have 21 bits of the 24), so that the gradient knows it.  The second
// condition takes no instruction a weight; counting what rounding takes of the value
// weights w 2^(e - E) too costs three, and registers that heads of 128 do not have (8192
// tokens below: 361 us for 290).
//
// Layout.  The matrix instruction's result holds one column per lane (column
// lane % 16, rows 4 (lane / 16) + r), its operands 16 consecutive steps of a
// contraction of 64 (steps 16 (lane / 16) ..).  Products run with the axis that
// is summed next (keys, for queries in the columns) along the rows: four results
// of 16 rows are then, lane by lane, the 16 bytes of the next product's operand
// for a contraction over their 64 rows, without a trip through LDS; that
// product's other operand takes its steps in the same order (frag_t).  Sixteen
// columns to a wave, not 32: a wave's sums take half the registers, which is
// two to four waves to a SIMD where there was one.
#pragma once

#include "ie_attn_index.h"
#include "ie_f64.h"
#include "ie_internal.h"

#pragma clang fp contract(off)

namespace ie {

constexpr int ATT_E_LO = -126, ATT_E_HI = 16;  // exponents of fp32's normal numbers
constexpr int CACHE_E_HI = ATT_E_HI + 5;  // 8-bit mantissas in 4 bits: the largest, 128, is 4 2^5
constexpr float W_C3 = 2545.0f * 0x1p-32f, W_C2 = 7358.0f * 0x1p-32f, W_C1 = 22609.0f * 0x1p-32f,
                W_C0 = 32512.0f * 0x1p-32f;
constexpr float RINT_MAGIC = 12582912.0f;  // 1.5 * 2^23: a sum's low bits are a whole number
constexpr int RINT_BITS = 0x4B400000;
constexpr float RINT_128 = RINT_MAGIC + 128.0f;
constexpr int ATT_CHECK = 2032, ATT_FINE = 14;
constexpr float FINE_UNIT = 16384.0f;  // 2^ATT_FINE
constexpr int16_t P_FINE = -31000;     // in the place of a need: the head's fine weights are still to be taken
constexpr int FINE_WORD = 8;           // of the workspace's header: whether there is such a head; zero between calls

__device__ __forceinline__ int clip_e(int e, int most = ATT_E_HI) { return min(max(e, ATT_E_LO), most); }
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ float pow2_down(int e) { return pow2f(max(e, -126)); }        // e <= 0: what is less rounds to 0

// The polynomial's coefficients, times a power of two where a row has one.
struct Poly {
    float c3, c2, c1, c0;
};
__device__ __forceinline__ Poly poly(float s) { return Poly{W_C3 * s, W_C2 * s, W_C1 * s, W_C0 * s}; }

// 32512 * 2^(d r), see above (d <= 0).
__device__ __forceinline__ float weight(float d, float r, const Poly &c = Poly{W_C3, W_C2, W_C1, W_C0}) {
    const float z = fmaxf(__builtin_fmaf(d, r, 96.0f), 64.0f);
    const float f = __builtin_amdgcn_fractf(z);
    uint32_t k;  // as written, the compiler takes the field's place by a shift and a mask
    asm("v_bfe_u32 %0, %1, 17, 6" : "=v"(k) : "v"(z));
    float q = __builtin_fmaf(c.c3, f, c.c2);
    q = __builtin_fmaf(q, f, c.c1);
    q = __builtin_fmaf(q, f, c.c0);
    return __int_as_float((int)(k << 23) + __float_as_int(q));
}

// The digits of four n + 128 in the low halves of a..d: high digits and low
// digits, a byte each.
__device__ __forceinline__ void digits4(int a, int b, int c, int d, int &hi, int &lo) {
    const uint32_t s = __builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x05010400u);
    const uint32_t t = __builtin_amdgcn_perm((uint32_t)d, (uint32_t)c, 0x05010400u);
    lo = (int)(__builtin_amdgcn_perm(t, s, 0x05040100u) ^ 0x80808080u);
    hi = (int)__builtin_amdgcn_perm(t, s, 0x07060302u);
}

// Three digits of four n + 0x8080 + 2^22 in the low 23 bits, |n| < 2^21.
__device__ __forceinline__ void digits3x4(int a, int b, int c, int d, int &hi, int &mid, int &lo) {
    digits4(a, b, c, d, mid, lo);
    mid ^= (int)0x80808080u;
    const uint32_t s = __builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x0c0c0602u);
    const uint32_t t = __builtin_amdgcn_perm((uint32_t)d, (uint32_t)c, 0x0c0c0602u);
    // bytes 64 + h, h from -32 to 32: no byte borrows from the next
    hi = (int)(((__builtin_amdgcn_perm(t, s, 0x05040100u) | 0x80808080u) - 0x40404040u) ^ 0x80808080u);
}

// Four digits of four n: of the highest bytes on, a word of four bytes each.
__device__ __forceinline__ void digits4x4(const int (&n)[4], int (&out)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = (uint32_t)n[i] + 0x808080u;
    const uint32_t s = __builtin_amdgcn_perm(u[1], u[0], 0x05010400u), t = __builtin_amdgcn_perm(u[3], u[2], 0x05010400u);
    const uint32_t v = __builtin_amdgcn_perm(u[1], u[0], 0x07030602u), w = __builtin_amdgcn_perm(u[3], u[2], 0x07030602u);
    out[0] = (int)__builtin_amdgcn_perm(w, v, 0x07060302u);
    out[1] = (int)(__builtin_amdgcn_perm(w, v, 0x05040100u) ^ 0x80808080u);
    out[2] = (int)(__builtin_amdgcn_perm(t, s, 0x07060302u) ^ 0x80808080u);
    out[3] = (int)(__builtin_amdgcn_perm(t, s, 0x05040100u) ^ 0x80808080u);
}
__device__ __forceinline__ double whole4(int a, int b, int c, int d) {
    return __builtin_fma(__builtin_fma(__builtin_fma((double)a, 256.0, (double)b), 256.0, (double)c), 256.0, (double)d);
}

__device__ __forceinline__ v4i mfma(v4i a, v4i b, v4i c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0); }

// A maximum over the four lanes of a column.
__device__ __forceinline__ float col_max(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
template <class F>
__device__ __forceinline__ int col_reduce(int v, F f) {
    return swap_reduce<32>(swap_reduce<16>(v, f), f);
}

template <bool B>
struct Bool {
    static constexpr bool value = B;
};

// The lanes of a wave, as the search for a tile uses them (ie_attn_index.h).
struct WaveLanes {
    using Int = int;
    template <class F>
    __device__ __forceinline__ int each(F f) const { return f((int)(threadIdx.x & 63)); }
    template <class F>
    __device__ __forceinline__ uint64_t ballot(F f) const { return __ballot(f((int)(threadIdx.x & 63))); }
    __device__ __forceinline__ int of(int x, int) const { return x; }
    __device__ __forceinline__ int at(int x, int lane) const { return __builtin_amdgcn_readlane(x, lane); }
    __device__ __forceinline__ int sum(int x) const { return __builtin_amdgcn_readfirstlane(lane_reduce<64>(x, Add{})); }
    __device__ __forceinline__ int max(int x) const { return wave_max_dpp(x); }
};
__device__ __forceinline__ Item att_item(const AttnArgs &p, int per) { return att_item(p, per, (int)blockIdx.x, (int)gridDim.x); }
template <bool HEAVY>
__device__ __forceinline__ bool rank_tile(const AttnArgs &p, int rank, int bm, Span &sp, int &tile) {
    return rank_tile<HEAVY>(WaveLanes{}, p, rank, bm, sp, tile);
}
inline int att_chunk(const AttnArgs &a, int bm, bool alike) { return att_chunk(a.rows, a.n_seq, a.kv, bm, alike && a.off); }

// 16 mantissas of a head from column 16 c on, at any alignment; past d: zeros.
__device__ __forceinline__ v4i head16(const int8_t *head, int c, int d) {
    v4i v = {0, 0, 0, 0};
    const int n = d - 16 * c;
    const int8_t *p = head + 16 * c;
    if (n >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else if (n > 0) {
        // n = 8 a + 4 b + 2 c + e, from the top down: each piece shifts the ones above it up
        uint64_t lo = 0, hi = 0;
        if (n & 8) __builtin_memcpy(&lo, p, 8);
        const int8_t *t = p + (n & 8);
        uint64_t w = 0;
        if (n & 1) w = (uint8_t)t[n & 6];
        if (n & 2) {
            uint16_t x;
            __builtin_memcpy(&x, t + (n & 4), 2);
            w = w << 16 | x;
        }
        if (n & 4) {
            uint32_t x;
            __builtin_memcpy(&x, t, 4);
            w = w << 32 | x;
        }
        if (n & 8) hi = w;
        else lo = w;
        v = v4i{(int)(uint32_t)lo, (int)(uint32_t)(lo >> 32), (int)(uint32_t)hi, (int)(uint32_t)(hi >> 32)};
    }
    return v;
}

// A tile of 64 rows of one head in LDS, read by rows (frag_r: contraction over
// the head's elements, 64 a step, zeros past its end) and transposed (frag_t).  Rows
// lie 16 bytes more than a multiple of 64 apart, and every 16 rows another 128
// bytes: the 16 rows of a frag_r, and the rows 4 c .. 4 c + 3 and 16 + 4 c .. of
// two lane groups of a frag_t, then fall on banks of their own (without the 128
// bytes 41 % of the cycles of LDS were conflicts, with them 30 %; the time is the
// same).
//
// Loads go through a buffer descriptor over the tile's rows, whose bounds are
// checked in hardware: a thread's chunks keep their offsets from tile to tile
// (rows past the last one and columns past the head lie outside it and read zeros),
// and only the descriptor, in scalar registers, moves.
// NT threads share the work: a workgroup, or a wave for a tile of its own.
template <int DP, int NT = 256>
struct HeadTile {
    static constexpr int KS = (DP + 63) / 64, CH = 4 * KS, PITCH = 64 * KS + 16, BYTES = 64 * PITCH + 3 * 128;
    static constexpr int NPT = (64 * CH + NT - 1) / NT;
    v4i reg[NPT];
    uint32_t at[NPT];
    __device__ __forceinline__ void init(long long width, int dp) {
#pragma unroll
        for (int i = 0; i < NPT; ++i) {
            const int c = threadIdx.x % NT + NT * i;
            const bool on = c < 64 * CH && c % CH * 16 < dp;
            at[i] = on ? (uint32_t)(c / CH) * (uint32_t)width + c % CH * 16 : 0x80000000u;
        }
    }
    // rows first .. of the head whose row 0 is at `head`, `n` rows in all
    __device__ __forceinline__ void fetch(const int8_t *head, long long width, int first, int n, int dp) {
        const uint64_t a = (uint64_t)(head + first * width);
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
        const int left = min(64, n - first);  // a tile behind the last row: no bytes
        const int bytes = __builtin_amdgcn_readfirstlane(left > 0 ? (left - 1) * (int)width + dp : 0);
        const auto r = __builtin_amdgcn_make_buffer_rsrc((void *)(((uint64_t)hi << 32) | lo), (short)0, bytes, 0x00020000);
#pragma unroll
        for (int i = 0; i < NPT; ++i) reg[i] = (v4i)__builtin_amdgcn_raw_buffer_load_b128(r, (int)at[i], 0, 0);
    }
    __device__ __forceinline__ void put(int8_t *lds) const {
#pragma unroll
        for (int i = 0; i < NPT; ++i) {
            const int c = threadIdx.x % NT + NT * i;
            if (64 * CH % NT && c >= 64 * CH) continue;
            *(v4i *)(lds + c / CH * PITCH + c / CH / 16 * 128 + c % CH * 16) = reg[i];
        }
    }
    // Rows 16 t .. as an operand: contraction over the head's elements 64 s ..
    static __device__ __forceinline__ v4i frag_r(const int8_t *lds, int t, int s, int lane) {
        return *(const v4i *)(lds + (lane & 15) * PITCH + t * (16 * PITCH + 128) + s * 64 + (lane >> 4) * 16);
    }
    // Elements 16 e .. as rows of an operand: contraction over the tile's 64
    // rows, in the order of the products' results (lane group c, byte 4 t + r:
    // row 16 t + 4 c + r).
    static __device__ __forceinline__ v4i frag_t(const int8_t *lds, int e, int lane) {
        const int g = lane & 15, k = g >> 1;
        const int8_t *at = lds + (4 * (lane >> 4) + (k & 3)) * PITCH + (k >> 2) * (16 * PITCH + 128) + 16 * e + (g & 1) * 8;
        typedef __attribute__((address_space(3))) v2i lds_v2i;
        const v2i lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)at);
        const v2i hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(at + 2 * (16 * PITCH + 128)));
        return v4i{lo.x, lo.y, hi.x, hi.y};
    }
};

// The head of a row as the operand that stays in registers: lane l holds row l
// % 16, elements 64 s + 16 (l / 16) ...
template <int KS>
__device__ __forceinline__ void head_regs(const int8_t *head, bool ok, int dp, int lane, v4i (&q)[KS]) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        q[s] = v4i{0, 0, 0, 0};
        const int c = 64 * s + (lane >> 4) * 16;
        if (ok && c < dp) q[s] = *(const v4i *)(head + c);
    }
}

// Sums of four waves into the first one's (exact integers), through LDS.
template <int N>
__device__ __forceinline__ void gather_waves(int *x, v4i (&acc)[N / 4], int wave, int lane) {
    __syncthreads();
    if (wave)
#pragma unroll
        for (int i = 0; i < N; ++i) x[((wave - 1) * N + i) * 64 + lane] = acc[i >> 2][i & 3];
    __syncthreads();
    if (!wave)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i >> 2][i & 3] += x[i * 64 + lane] + x[(N + i) * 64 + lane] + x[(2 * N + i) * 64 + lane];
}

// Results of one head, columns of a transposed product: value y[4 g + r] of lane
// l is element 16 e_g + 4 (l / 16) + r of row l % 16; the other three quarters of
// these elements lie 16, 32 and 48 lanes away.  They are rounded to odd at two
// bits below what the head alone needs, for a rounding by whole rows.
template <int NV>
__device__ __forceinline__ int max_word(const double (&y)[NV]) {
    MaxMag mx;
#pragma unroll
    for (int i = 0; i < NV; i += 2) mx.add(y[i], y[i + 1]);
    return col_reduce(mx.word(), Max{});
}
__device__ __forceinline__ void write_odd(const double *y, double inv, bool ok, int c, int d, int16_t *out) {
    int v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const double t = y[k] * inv, f = floor(t);
        v[k] = (int)f | (f != t ? 1 : 0);
    }
    if (!ok) return;
    if (d % 4 == 0) {
        if (c < d) *(int2 *)(out + c) = int2{(v[0] & 0xffff) | v[1] << 16, (v[2] & 0xffff) | v[3] << 16};
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c + k < d) out[c + k] = (int16_t)v[k];
    }
}
__device__ __forceinline__ double odd_scale(int need) { return need == NEED_NONE ? 0.0 : pow2(2 - need); }
template <int NV>
__device__ __forceinline__ void store_odd(const double (&y)[NV], int e, int q, bool ok, int d, int lane, int16_t *out,
                                          int16_t *need_out) {
    const int need = need_word(max_word(y), q);
    const double inv = odd_scale(need);
    if (ok && lane < 16) *need_out = (int16_t)(need == NEED_NONE ? P_NONE : need + e);
#pragma unroll
    for (int g = 0; g < NV / 4; ++g) write_odd(y + 4 * g, inv, ok, 16 * g + 4 * (lane >> 4), d, out);
}

}  // namespace ie
