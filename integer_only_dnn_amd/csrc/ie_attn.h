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
// seven.  The unit resolution of 2^-17 and the polynomial's error are an
// order below half a step of the 7-bit mantissas that come out.
//
// Digits.  A weight enters a product as an integer n = rint(w ...) of at most
// 32512, as two signed digits n = 256 a + b, a and b int8, so that its sums
// are exact int32 sums of v_mfma_i32_32x32x32_i8 and the order of keys, of
// tiles and of workgroups is of no account.  n + 128 comes out of the adder of
// rint (a magic constant), its two low bytes are a and b + 128.
//
// Layout.  The matrix instruction's result holds one column per lane (column
// lane % 32, rows 8 (r / 4) + 4 (lane / 32) + r % 4), its operands 16
// consecutive steps of the contraction.  Products run with the axis that is
// summed next (keys, for queries in the columns) along the rows: four
// neighbouring results of a lane are then four neighbouring bytes of the next
// product's operand, without a trip through LDS; the other operand of that
// product takes its steps in the same order (frag_t).
#pragma once

#include "ie_f64.h"
#include "ie_internal.h"

#pragma clang fp contract(off)

namespace ie {

constexpr int ATT_E_LO = -48, ATT_E_HI = 16;
constexpr float W_C3 = 2545.0f * 0x1p-32f, W_C2 = 7358.0f * 0x1p-32f, W_C1 = 22609.0f * 0x1p-32f,
                W_C0 = 32512.0f * 0x1p-32f;
constexpr float RINT_MAGIC = 12582912.0f;  // 1.5 * 2^23: a sum's low bits are a whole number
constexpr int RINT_BITS = 0x4B400000;
constexpr float RINT_128 = RINT_MAGIC + 128.0f;

__device__ __forceinline__ int clip_e(int e) { return min(max(e, ATT_E_LO), ATT_E_HI); }
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// 32512 * 2^(d r), see above (d <= 0).
__device__ __forceinline__ float weight(float d, float r) {
    const float z = fmaxf(__builtin_fmaf(d, r, 96.0f), 64.0f);
    const float f = __builtin_amdgcn_fractf(z);
    const uint32_t k = (uint32_t)__float_as_int(z) >> 17 & 63u;
    float q = __builtin_fmaf(W_C3, f, W_C2);
    q = __builtin_fmaf(q, f, W_C1);
    q = __builtin_fmaf(q, f, W_C0);
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

// Three digits of four n + 0x8080 + 2^22 in the low 23 bits, |n| < 2^21: high
// ones 64 too large, middle and low ones.
__device__ __forceinline__ void digits3x4(int a, int b, int c, int d, int &hi, int &mid, int &lo) {
    digits4(a, b, c, d, mid, lo);
    mid ^= (int)0x80808080u;
    const uint32_t s = __builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x0c0c0602u);
    const uint32_t t = __builtin_amdgcn_perm((uint32_t)d, (uint32_t)c, 0x0c0c0602u);
    hi = (int)__builtin_amdgcn_perm(t, s, 0x05040100u);
}

__device__ __forceinline__ v16i mfma(v4i a, v4i b, v16i c) { return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0); }

__device__ __forceinline__ float half_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Sequence s of a packed batch: its rows [a, b).  Offsets are read on the
// device; bounds that lie outside the matrix or before the last one are
// clipped, a sequence longer than `most` is cut there.
struct Span {
    int a, n;
};
__device__ __forceinline__ Span seq_span(const AttnArgs &p, int s) {
    if (!p.off) return Span{0, (int)min(p.rows, (long long)p.most)};
    const int rows = (int)p.rows;
    const int a = min(max(p.off[s], 0), rows), b = min(max(p.off[s + 1], a), rows);
    return Span{a, min(b - a, p.most)};
}
// Tiles of BM rows: sequence s owns the slots from off[s] / BM + s on, enough
// for its ceil(n / BM) tiles whatever the other lengths are, so that a slot
// finds its sequence by bisection and nothing is laid out beforehand.  Returns
// the sequence's rows and the tile's first row in it (>= n: no such tile).
__device__ __forceinline__ Span slot_span(const AttnArgs &p, int slot, int bm, int &first, int &seq) {
    seq = 0;
    if (!p.off) {
        first = slot * bm;
        return seq_span(p, 0);
    }
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (max(p.off[mid], 0) / bm + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    seq = lo;
    const Span s = seq_span(p, lo);
    const int at = slot - (max(p.off[lo], 0) / bm + lo);
    first = at < 0 || at > s.n / bm ? s.n : at * bm;
    return s;
}

// Work items (tile slots of every head) as workgroups reach the XCDs
// (blockIdx % 8): each XCD takes a contiguous run, so that the tiles and the
// query heads that share keys share its L2.  -1: none.
__device__ __forceinline__ long long xcd_item(long long total) {
    const long long per = (total + 7) / 8, i = (long long)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    return (blockIdx.x >> 3) < per && i < total ? i : -1;
}

// 16 mantissas of a head from column 16 c on; past d: zeros.
__device__ __forceinline__ v4i head16(const int8_t *head, int c, int d, int vec) {
    v4i v = {0, 0, 0, 0};
    const int n = d - 16 * c;
    if (n <= 0) return v;
    if (vec) return *(const v4i *)(head + 16 * c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 16; ++k)
        if (k < n) w[k >> 2] |= (uint32_t)(uint8_t)head[16 * c + k] << (8 * (k & 3));
    return v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// A tile of 64 rows of one head, DP bytes each (zeros past d), in LDS: read by
// rows (frag_r) and transposed (frag_t).  Rows lie DP + PAD bytes apart, which
// spreads the 16-byte reads of 32 rows and the eight rows of a transposing
// read over the banks.
template <int DP>
struct HeadTile {
    static constexpr int CH = DP / 16, PITCH = DP + (DP == 32 ? 16 : DP == 64 ? 16 : 16), BYTES = 64 * PITCH;
    static constexpr int NPT = (64 * CH + 255) / 256;
    v4i reg[NPT];
    // rows first .. of the head whose row 0 is at `head`, `n` rows in all
    __device__ __forceinline__ void fetch(const int8_t *head, long long width, int first, int n, int d, int vec) {
#pragma unroll
        for (int i = 0; i < NPT; ++i) {
            const int c = threadIdx.x + 256 * i, row = c / CH;
            reg[i] = v4i{0, 0, 0, 0};
            if (64 * CH % 256 && c >= 64 * CH) continue;
            if (first + row < n) reg[i] = head16(head + (first + row) * width, c % CH, d, vec);
        }
    }
    __device__ __forceinline__ void put(int8_t *lds) const {
#pragma unroll
        for (int i = 0; i < NPT; ++i) {
            const int c = threadIdx.x + 256 * i;
            if (64 * CH % 256 && c >= 64 * CH) continue;
            *(v4i *)(lds + c / CH * PITCH + c % CH * 16) = reg[i];
        }
    }
    // Rows row .. row + 31 as an operand whose contraction is the head's
    // elements 32 s ..: lane l holds row l % 32.
    static __device__ __forceinline__ v4i frag_r(const int8_t *lds, int row, int s, int lane) {
        return *(const v4i *)(lds + (row + (lane & 31)) * PITCH + s * 32 + (lane >> 5) * 16);
    }
    // Elements 32 s .. as rows of an operand whose contraction are the tile's
    // rows row .. row + 31, in the order of a product's results.
    static __device__ __forceinline__ v4i frag_t(const int8_t *lds, int row, int s, int lane) {
        const int g = lane & 15, k = g >> 1;
        const int8_t *at = lds + (row + (k >> 2) * 8 + (lane >> 5) * 4 + (k & 3)) * PITCH + s * 32 + (lane & 16) + (g & 1) * 8;
        typedef __attribute__((address_space(3))) v2i lds_v2i;
        const v2i lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)at);
        const v2i hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(at + 16 * PITCH));
        return v4i{lo.x, lo.y, hi.x, hi.y};
    }
};

// The head of a row as the operand that stays in registers: lane l holds row
// l % 32, elements 32 s + 16 (l / 32) ...
template <int DP>
__device__ __forceinline__ void head_regs(const int8_t *head, bool ok, int d, int vec, int lane, v4i (&q)[DP / 32]) {
#pragma unroll
    for (int s = 0; s < DP / 32; ++s) {
        q[s] = v4i{0, 0, 0, 0};
        if (ok) q[s] = head16(head, 2 * s + (lane >> 5), d, vec);
    }
}

// A result row of one head, one column of the transposed product: value
// y[16 s + r] of lane l is element 32 s + 8 (r / 4) + 4 (l / 32) + r % 4 of row
// l % 32; the other half of the row lies in the lane 32 away.  Rounded to odd
// at two bits below what the head alone needs, for a rounding by whole rows.
template <int NV>
__device__ __forceinline__ void store_odd(const double (&y)[NV], int e, int q, bool ok, int d, int lane, int16_t *out,
                                          int16_t *need_out) {
    MaxMag mx;
#pragma unroll
    for (int i = 0; i < NV; i += 2) mx.add(y[i], y[i + 1]);
    const int need = need_word(swap_reduce<32>(mx.word(), Max{}), q);
    const double inv = need == NEED_NONE ? 0.0 : pow2(2 - need);
    if (ok && lane < 32) *need_out = (int16_t)(need == NEED_NONE ? P_NONE : need + e);
#pragma unroll
    for (int g = 0; g < NV / 4; ++g) {
        const int c = 32 * (g / 4) + 8 * (g % 4) + 4 * (lane >> 5);
        int v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const double t = y[4 * g + k] * inv, f = floor(t);
            v[k] = (int)f | (f != t ? 1 : 0);
        }
        if (!ok) continue;
        if (d % 4 == 0) {
            if (c < d) *(int2 *)(out + c) = int2{(v[0] & 0xffff) | v[1] << 16, (v[2] & 0xffff) | v[3] << 16};
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + k < d) out[c + k] = (int16_t)v[k];
        }
    }
}

}  // namespace ie
