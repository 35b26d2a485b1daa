// Keys and values of 4-bit mantissas in a paged cache, and attention of single
// tokens over it.
//
// A slot of the cache holds, for every key head, head_dim mantissas of 4 bits
// (|C| <= 7) with one exponent for the key and one for the value; two
// mantissas to a byte, the even one in the low half.
#include "ie_attn.h"

#pragma clang fp contract(off)

namespace ie {

constexpr int CACHE_CHECK = 8;  // blocks whose weights are rounded without a check
constexpr int STORE_ROWS = 4096;  // numbers of a chunk's heads fit 30 bits

// One key or value head of a row: NL lanes with 16 mantissas each.  8192 rows of 8
// heads of 128 (25 MB) in 9 us; 16 rows in 3.3 us, a launch's time.
template <int NL>
__global__ __launch_bounds__(256) void cache_store_kernel(CacheArgs p, long long rows, const int8_t *x, const int8_t *xe, int x_row,
                                                          int width, int first, const int *slots, FastDiv by_parts) {
    constexpr int PB = 256 / NL;
    const int parts = 2 * p.kv, lane = threadIdx.x % NL;
    const long long slot_max = (long long)p.pages * p.page;
    for (long long row0 = (long long)blockIdx.y * STORE_ROWS; row0 < rows; row0 += (long long)gridDim.y * STORE_ROWS)
    for (int i0 = blockIdx.x * PB, total = (int)min(rows - row0, (long long)STORE_ROWS) * parts; i0 < total; i0 += gridDim.x * PB) {
        const int i = min(i0 + (int)threadIdx.x / NL, total - 1);
        const int r = (int)(((uint64_t)(uint32_t)i * by_parts.m) >> by_parts.s), part = i - r * parts;
        const long long row = row0 + r, slot = slots[row];
        const bool mine = i == i0 + (int)threadIdx.x / NL, on = mine && slot >= 0 && slot < slot_max;
        if (mine && slot >= slot_max && lane == 0) atomicOr(p.flags, IE_FLAG_INDEX);
        uint32_t w[4] = {0, 0, 0, 0};
        const bool have = on && 16 * lane < p.d;
        if (have) __builtin_memcpy(w, x + row * width + first + part * p.d + 16 * lane, 16);
        const int ex = xe[x_row ? row : 0];
        int m = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) m = max(m, abs(byte_of(w[k >> 2], k & 3)));
        m = lane_reduce<NL>(m, Max{});
        const int e = max(E_MIN, need32(m, ex, 3));
        // C 2^(ex - e) rounded: exact products, at most 7.5
        const float inv = __int_as_float((127 + min(max(ex - e, -100), 100)) << 23);
        uint32_t o[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 16; ++k)
            o[k >> 3] |= ((uint32_t)__float_as_int(__builtin_fmaf((float)byte_of(w[k >> 2], k & 3), inv, RINT_MAGIC)) & 15u) << (4 * (k & 7));
        if (!on) continue;
        const bool val = part >= p.kv;
        const long long at = slot * p.kv + (val ? part - p.kv : part);
        if (lane == 0) (val ? p.ve : p.ke)[at] = (int8_t)clamp_exp_flag(e, p.flags);
        if (have) *(uint2 *)((val ? p.v : p.k) + at * (p.d >> 1) + 8 * lane) = uint2{o[0], o[1]};
    }
}

// Attention of one token a sequence.  Keys are taken in blocks of 256 of a
// sequence's positions; a block b has its own maximum m_b and value exponent
// E_b, and sums of integers as in attention over a prompt:
//   L_b = sum R(w_j),  N_b = sum R(w_j 2^(ev_j - E_b)) v_j;
// a block enters the whole with the weight of its maximum, another such
// integer: a_b = W(m_b - m),  L = sum R(a_b) L_b,  E = max E_b,
//   o = (sum R(a_b 2^(E_b - E)) N_b) (1 / L) 2^E
// (in finer units where that rounding takes too much, see cache_join_kernel).
// All sums are exact (in 64 bits: 2^23 keys with values of 8 units come to 32512^2 2^26 <
// 2^56), so that how blocks are shared out is of no account, and each key and
// value is read once.
//
// A workgroup takes a block of one key head and up to 16 of its query heads,
// a wave 64 of the keys: 16x16x64 products with the keys along the rows and
// the query heads in the columns.  Where eight or four columns are enough for
// the heads, each head has SUB of them, and each of those weighs its share of
// the wave's keys.  The weights' digits change hands in LDS, and a wave sums
// 32 (DP 64: 16) of the elements over all keys.  Values lie in LDS as they
// come, two elements to a byte: a transposing read of 16 columns of bytes is
// unpacked into two operands, the even elements and the odd ones.  Mantissas
// are unpacked as 16 times their value (their four bits in a byte's upper half),
// which the exact sums drop.  The next block's keys, values and exponents and the
// slots of the one behind it are in flight while one is computed.
//
// 48 sequences of up to 8000 tokens, 32 heads on 8 of 128 (196 MB) 45 us where the cache's
// last level holds them, 4.3 TB/s, and 60 from memory; one of 131072 (136 MB) 32 and 42.
// Waits are 56 % of a wave's life, vector instructions 48 % of the busy cycles: neither the
// stream nor the instructions alone.  A key head's 64 bytes are half a line, whose
// other half another workgroup reads.  SUB 1 for these four heads takes 5 % longer.
template <int SUB>
__device__ __forceinline__ float heads_max(float v) {
    v = col_max(v);
    if (SUB > 1) v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 15, 15, true)));
    if (SUB > 2) v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 15, 15, true)));
    return v;
}
template <int SUB>
__device__ __forceinline__ int heads_sum(int v) {
    v = col_reduce(v, Add{});
    if (SUB > 1) v += __builtin_amdgcn_update_dpp(0, v, 0x128, 15, 15, true);
    if (SUB > 2) v += __builtin_amdgcn_update_dpp(0, v, 0x124, 15, 15, true);
    return v;
}
template <int DP, int SUB>  // head size, up: 64 or 128
__global__ __launch_bounds__(256, 4) void cache_attention_kernel(CacheArgs p, AttnArgs a) {
    constexpr int NS = DP / 64, PITCH = DP / 2 + 16, HC = 16 / SUB, TN = 4 / SUB;
    __shared__ __align__(16) int8_t sv[256 * PITCH];
    __shared__ __align__(16) float sfk[256], sfv[256];
    __shared__ __align__(16) int sdigit[2][4][16][4][4];  // high and low: wave, head, keys 4 c .., 16 t ..
    __shared__ __align__(16) int scum[256];
    __shared__ int slen[256], swave[4], sred[4], ssum[4][16];
    __shared__ float smax[4][16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, c = lane >> 4;
    const int hc = col & (HC - 1), tp = col / HC * TN;  // head of the group, first 16 keys it weighs
    const int gcs = (a.group + 15) / 16, units = a.kv * gcs, hb = a.d >> 1;
    // Items: block b of a sequence, a key head and 16 of its query heads; in
    // groups of eight blocks, a block's heads eight apart: the heads of a slot
    // share cache lines, and these workgroups an XCD.  A workgroup's items lie
    // gridDim (a multiple of 8) apart.
    const unsigned turn = gridDim.x >> 3;
    const int by_q = (int)turn / units, by_u = (int)turn % units, r8 = blockIdx.x & 7;
    unsigned before = 0;
    int s0 = 0, blocks = 0;  // sequences s0 .. s0 + 255 and their blocks of 256 keys
    struct Work {
        int q, unit;  // blocks 8 q .., key head and its query heads
        int seq, b, kvh, g0, len;
    };
    auto advance = [&](Work &w) {
        w.q += by_q;
        w.unit += by_u;
        if (w.unit >= units) {
            w.unit -= units;
            ++w.q;
        }
    };
    auto locate = [&](Work &w) {  // the first item from (q, unit) on that there is
        while (8 * w.q < blocks) {
            const int blk = 8 * w.q + r8;
            if (blk < blocks) {
                const int4 x = ((const int4 *)scum)[lane];
                const int i = __popcll(__ballot(x.x <= blk)) + __popcll(__ballot(x.y <= blk)) + __popcll(__ballot(x.z <= blk)) +
                              __popcll(__ballot(x.w <= blk));
                w.seq = s0 + i;
                w.b = blk - __builtin_amdgcn_readfirstlane(i ? scum[i - 1] : 0);
                w.kvh = gcs == 1 ? w.unit : w.unit / gcs;
                w.g0 = (w.unit - w.kvh * gcs) * 16;
                w.len = __builtin_amdgcn_readfirstlane(slen[i]);
                return true;
            }
            advance(w);
        }
        return false;
    };
    auto slot_of = [&](const Work &w) {  // of key 256 b + tid
        const int j = 256 * w.b + tid;
        if (j >= w.len) return -1;
        const int page = p.table[(long long)w.seq * p.per + (j >> p.shift)];
        return page >= 0 && page < p.pages ? (page << p.shift) + (j & (p.page - 1)) : -2;
    };
    // what is read of a block: lane (col, c) takes 16 bytes (DP 64: 8) of the
    // wave's keys col, 16 + col, ..; thread t the exponents of key t
    uint32_t kw[4][2 * NS], vw[4][2 * NS];
    float fk = 0.0f, fv = 0.0f;
    auto take = [&](const Work &w, int mine, const auto *from, uint32_t (&to)[4][2 * NS]) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int slot = __shfl(mine, 16 * t + col, 64);
            const long long at = ((long long)slot * p.kv + w.kvh) * hb + 8 * NS * c;
#pragma unroll
            for (int i = 0; i < 2 * NS; ++i) to[t][i] = 0;
            if (slot < 0) continue;
            if (8 * NS * (c + 1) <= hb) __builtin_memcpy(to[t], from + at, 8 * NS);
            else if (8 * NS * c < hb) __builtin_memcpy(to[t], from + at, 8);
        }
    };
    auto fetch_keys = [&](const Work &w, int mine) {
        fk = fv = 0.0f;
        if (mine >= 0) {
            const long long at = (long long)mine * p.kv + w.kvh;
            const int ek = p.ke[at], ev = p.ve[at];
            fk = pow2f(clip_e(ek, CACHE_E_HI));
            fv = pow2f(clip_e(ev, CACHE_E_HI));
            if (max(ek, ev) > CACHE_E_HI) atomicOr(p.flags, IE_FLAG_EXP_RANGE);
        }
        if (mine == -2) atomicOr(p.flags, IE_FLAG_INDEX);
        take(w, mine, p.k, kw);
    };

    for (s0 = 0; s0 < p.n; s0 += 256) {
        // blocks of the next 256 sequences, and their running sum
        const int len = s0 + tid < p.n ? min(max(p.lengths[s0 + tid], 0), p.tokens) : 0;
        int run = (len + 255) >> 8;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(run, o, 64);
            if (lane >= o) run += v;
        }
        __syncthreads();
        if (lane == 63) swave[wave] = run;
        __syncthreads();
        for (int i = 0; i < wave; ++i) run += swave[i];
        scum[tid] = run;
        slen[tid] = len;
        __syncthreads();
        blocks = __builtin_amdgcn_readfirstlane(scum[255]);
        const unsigned first = (blockIdx.x / 8 + turn - before) % turn;
        before = (before + (unsigned)((blocks + 7) / 8) % turn * ((unsigned)units % turn)) % turn;
        Work w;
        w.q = (int)first / units;
        w.unit = (int)first - w.q * units;
        // the item in hand (w) has its data on the way, the next one (ahead) its slots
        bool more = locate(w);
        if (more) {
            const int slot = slot_of(w);
            fetch_keys(w, slot);
            take(w, slot, p.v, vw);
        }
        Work ahead = w;
        auto look = [&]() {
            advance(ahead);
            return locate(ahead);
        };
        bool more_ahead = more && look();
        int slot = more_ahead ? slot_of(ahead) : -1;
        while (more) {
            const Work now = w;
            sfk[tid] = fk;
            sfv[tid] = fv;
            const int em = wave_max_dpp(__float_as_int(fv));
            if (lane == 0) sred[wave] = em;
            // the query heads, their bytes in the order of unpacked keys
            const int ng = min(HC, a.group - now.g0), head = now.kvh * a.group + now.g0 + hc;
            const float r = a.c * pow2f(clip_e(a.xe[a.x_row ? now.seq : 0]));
            v4i q[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                q[i] = v4i{0, 0, 0, 0};
                const int e0 = 16 * NS * c + 16 * i;
                if (hc < ng && e0 < a.d) {
                    uint32_t x[4];
                    __builtin_memcpy(x, a.x + (long long)now.seq * a.width + (long long)head * a.d + e0, 16);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        q[i][2 * z] = (int)__builtin_amdgcn_perm(x[2 * z + 1], x[2 * z], 0x06040200u);
                        q[i][2 * z + 1] = (int)__builtin_amdgcn_perm(x[2 * z + 1], x[2 * z], 0x07050301u);
                    }
                }
            }
            v4i acc[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                acc[t] = v4i{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    v4i k;
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        k[2 * z] = (int)(kw[t][2 * i + z] << 4 & 0xf0f0f0f0u);
                        k[2 * z + 1] = (int)(kw[t][2 * i + z] & 0xf0f0f0f0u);
                    }
                    acc[t] = mfma(k, q[i], acc[t]);
                }
            }
            float f[TN][4], m = -__builtin_inff();
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const float4 x = *(const float4 *)&sfk[64 * wave + 16 * (tp + j) + 4 * c];
                const float fs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    int s = acc[j][i];
                    if (SUB == 2) s = tp ? acc[2 + j][i] : s;
                    if (SUB == 4) s = tp & 2 ? (tp & 1 ? acc[3][i] : acc[2][i]) : (tp & 1 ? acc[1][i] : s);
                    f[j][i] = fs[i] > 0.0f ? (float)s * (0.0625f * fs[i]) : -__builtin_inff();
                    m = fmaxf(m, f[j][i]);
                }
            }
            if (more_ahead) fetch_keys(ahead, slot);
            m = heads_max<SUB>(m);
            if (lane < 16) smax[wave][lane] = m;
            __syncthreads();
            // values into LDS: every wave is past the last block's
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                int8_t *dst = sv + (64 * wave + 16 * t + col) * PITCH + 8 * NS * c;
                __builtin_memcpy(dst, vw[t], 8 * NS);
            }
            if (more_ahead) take(ahead, slot, p.v, vw);
            w = ahead;
            more = more_ahead;
            more_ahead = more && look();
            slot = more_ahead ? slot_of(ahead) : -1;
            const float fmx = __int_as_float(max(max(sred[0], sred[1]), max(sred[2], sred[3])));
            const int eb = fmx > 0.0f ? (__float_as_int(fmx) >> 23) - 127 : ATT_E_LO;
            const float down = pow2f(-eb);
            m = fmaxf(fmaxf(smax[0][col], smax[1][col]), fmaxf(smax[2][col], smax[3][col]));
            uint32_t sum = 0;
            int dh[TN], dl[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const float4 x = *(const float4 *)&sfv[64 * wave + 16 * (tp + j) + 4 * c];
                const float fvs[4] = {x.x, x.y, x.z, x.w};
                int bits[4];
                uint32_t whole_n[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a key that is not there: a score of minus infinity, whose weight rounds to 0, and a factor of 0
                    const float y = weight(f[j][i] - m, r);
                    bits[i] = __float_as_int(__builtin_fmaf(y, fvs[i] * down, RINT_128));
                    whole_n[i] = (uint32_t)__float_as_int(y + RINT_MAGIC);
                }
                sum += whole_n[0] + whole_n[1];
                sum += whole_n[2] + whole_n[3];
                digits4(bits[0], bits[1], bits[2], bits[3], dh[j], dl[j]);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                sdigit[0][wave][hc][c][tp + j] = dh[j];
                sdigit[1][wave][hc][c][tp + j] = dl[j];
            }
            sum = (uint32_t)heads_sum<SUB>((int)(sum - 4u * TN * (uint32_t)RINT_BITS));
            if (lane < HC) ssum[wave][lane] = (int)sum;
            __syncthreads();
            // the second product: rows are bytes' elements, even ones, then odd ones
            const int e = DP == 128 ? wave : wave >> 1;
            const bool upper = wave & 1;  // DP 64: the odd elements
            const long long out = ((long long)now.seq * p.blocks + now.b) * a.heads + now.kvh * a.group + now.g0;
            if (16 * e < hb) {
                v4i y[2][2] = {};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int g = lane & 15, kk = g >> 1;
                    const int8_t *at = sv + (64 * s + 16 * (kk >> 2) + 4 * c + (kk & 3)) * PITCH + 16 * e + (g & 1) * 8;
                    typedef __attribute__((address_space(3))) v2i lds_v2i;
                    const v2i x0 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)at);
                    const v2i x1 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(at + 32 * PITCH));
                    const uint32_t xs[4] = {(uint32_t)x0.x, (uint32_t)x0.y, (uint32_t)x1.x, (uint32_t)x1.y};
                    const v4i h4 = *(const v4i *)sdigit[0][s][hc][c], l4 = *(const v4i *)sdigit[1][s][hc][c];
                    v4i even, odd;
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        even[z] = (int)((DP == 64 && upper ? xs[z] : xs[z] << 4) & 0xf0f0f0f0u);
                        odd[z] = (int)(xs[z] & 0xf0f0f0f0u);
                    }
                    y[0][0] = mfma(even, h4, y[0][0]);
                    y[0][1] = mfma(even, l4, y[0][1]);
                    if (DP == 128) {
                        y[1][0] = mfma(odd, h4, y[1][0]);
                        y[1][1] = mfma(odd, l4, y[1][1]);
                    }
                }
                int *to = p.num + (out + hc) * a.d + 32 * e + 8 * c;
                if (col < ng && 32 * e + 8 * c < a.d) {
                    int x[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[2 * i] = (y[0][0][i] * 256 + y[0][1][i]) >> 4;
                        if (DP == 128) x[2 * i + 1] = (y[1][0][i] * 256 + y[1][1][i]) >> 4;
                        else to[2 * i + upper] = x[2 * i];
                    }
                    if (DP == 128) __builtin_memcpy(to, x, 32);
                }
            }
            if (tid < ng) {
                const int s = ssum[0][tid] + ssum[1][tid] + ssum[2][tid] + ssum[3][tid];
                p.top[out + tid] = int4{__float_as_int(m), s, eb, 0};
            }
        }
    }
}

// The blocks of one head of one sequence together, `piece` of its elements to a
// workgroup, as round-to-odd values and a need for a rounding by rows.  Blocks
// are taken 256 at a time: a thread finds the weights of one, then threads of
// four neighbouring elements add up a share of the blocks each.  Bound by its few
// round trips to memory: 8.7 us for the 21 MB of 48 sequences of up to 8000 tokens,
// 9.6 for one of 131072.
//
// Fine weights, as in attention over a prompt: a block's weight takes half a unit of
// its sums at most, of eight blocks (the largest's weight is exact) less than 7 * 128 /
// 32512 = 1 / 36 in all.  With more of them the weights' sum, and that of the values'
// weights a_b 2^(E_b - E), are taken in units of 2^-14 too; where that changes the first
// by more than a 32nd, or the second by so much that with values of 8 it is a fourth of
// the largest of 16 neighbouring elements, these elements are summed again in such units,
// in two halves of the weights.
__global__ __launch_bounds__(256) void cache_join_kernel(CacheArgs p, AttnArgs a, int piece) {
    __shared__ int sh[4];
    __shared__ int sw[256];
    __shared__ long long sp[256][4], sn[3][4];
    const int pieces = a.d / piece, tid = threadIdx.x;
    const int part_of = blockIdx.x % (a.heads * pieces), seq = blockIdx.x / (a.heads * pieces), head = part_of / pieces;
    const int len = min(max(p.lengths[seq], 0), p.tokens), nb = (len + 255) >> 8;
    if (tid == 0 && p.lengths[seq] != len) atomicOr(p.flags, IE_FLAG_INDEX);
    const int4 *top = p.top + (long long)seq * p.blocks * a.heads + head;
    const int *num = p.num + (long long)seq * p.blocks * a.cols + part_of * piece;
    float m = -__builtin_inff();
    int em = ATT_E_LO;
    for (int b = tid; b < nb; b += 256) {
        const int4 t = top[(long long)b * a.heads];
        if (t.y) {
            m = fmaxf(m, __int_as_float(t.x));
            em = max(em, t.z);
        }
    }
    // floats in the order of integers
    const int mi = __float_as_int(m), ordered = mi >= 0 ? mi : mi ^ 0x7fffffff;
    const int best = row_reduce<256>(ordered, Max{}, sh);
    em = row_reduce<256>(em, Max{}, sh);
    m = __int_as_float(best >= 0 ? best : best ^ 0x7fffffff);
    const float r = a.c * pow2f(clip_e(a.xe[a.x_row ? seq : 0]));
    const int quads = piece >> 2, parts = 256 / quads, part = tid / quads, e = 4 * (tid - part * quads);
    // one element's sum over the blocks (threads past the piece: 0), and sums of a thread's numbers of its blocks
    auto join = [&](auto weigh, long long (&n)[3]) {
        long long s[4] = {0, 0, 0, 0};
        n[0] = n[1] = n[2] = 0;
        for (int b0 = 0; b0 < nb; b0 += 256) {
            const int nc = min(256, nb - b0);
            __syncthreads();
            if (tid < nc) {
                const int4 t = top[(long long)(b0 + tid) * a.heads];
                sw[tid] = t.y ? weigh(weight(__int_as_float(t.x) - m, r), pow2_down(t.z - em), t.y, n) : 0;
            }
            __syncthreads();
            if (part < parts) {
#pragma unroll 4
                for (int b = part; b < nc; b += parts) {
                    int4 x;
                    __builtin_memcpy(&x, num + (long long)(b0 + b) * a.cols + e, 16);
                    const long long w = sw[b];
                    s[0] += w * x.x;
                    s[1] += w * x.y;
                    s[2] += w * x.z;
                    s[3] += w * x.w;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) sp[tid][k] = s[k];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            n[k] = lane_reduce<64>(n[k], Add{});
            if ((tid & 63) == 0) sn[k][tid >> 6] = n[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) n[k] = sn[k][0] + sn[k][1] + sn[k][2] + sn[k][3];
        long long sum = 0;
        if (tid < piece) {
#pragma unroll 8
            for (int i = 0; i < parts; ++i) sum += sp[i * quads + (tid >> 2)][tid & 3];
        }
        return sum;
    };
    long long n[3];  // the weights' sum, what rounding took of it in units of 2^-14, and of the values' weights
    const long long sum = join([](float x, float f, int l, long long (&n)[3]) {
        const int w = (int)__builtin_rintf(x), v = (int)__builtin_rintf(x * f);
        n[0] += (long long)w * l;
        n[1] += (long long)((int)__builtin_rintf(x * FINE_UNIT) - (w << ATT_FINE)) * l;
        n[2] += (long long)((int)__builtin_rintf(x * f * FINE_UNIT) - (v << ATT_FINE)) * l;
        return v;
    }, n);
    double y = n[0] > 0 ? (double)sum * (1.0 / (double)n[0]) : 0.0;
    const long long big = lane_reduce<16>(sum < 0 ? -sum : sum, [](long long x, long long z) { return x > z ? x : z; });
    // 512 = 2^14 / 32; 512 big may not fit 64 bits
    const bool much = (n[1] < 0 ? -n[1] : n[1]) > 512 * n[0] || ((n[2] < 0 ? -n[2] : n[2]) + 511) >> 9 > big;
    const bool fine = nb > CACHE_CHECK && n[0] > 0 && much && tid < piece;
    constexpr int SOME = 0x7fffffff;  // no result has such a high word
    int word = row_reduce<256>(fine ? SOME : __double2hiint(y) & 0x7fffffff, Max{}, sh);
    if (word == SOME) {
        long long hi_n[3], lo_n[3];
        const long long hi = join([](float x, float f, int l, long long (&n)[3]) {
            n[0] += (long long)((int)__builtin_rintf(x * FINE_UNIT) >> 15) * l;
            return (int)__builtin_rintf(x * f * FINE_UNIT) >> 15;
        }, hi_n);
        const long long lo = join([](float x, float f, int l, long long (&n)[3]) {
            n[0] += (long long)((int)__builtin_rintf(x * FINE_UNIT) & 32767) * l;
            return (int)__builtin_rintf(x * f * FINE_UNIT) & 32767;
        }, lo_n);
        if (fine) y = ((double)hi * 32768.0 + (double)lo) * (1.0 / ((double)hi_n[0] * 32768.0 + (double)lo_n[0]));
        word = row_reduce<256>(__double2hiint(y) & 0x7fffffff, Max{}, sh);
    }
    const int need = need_word(word, a.q);
    const long long at = (long long)seq * a.heads * pieces + part_of;
    if (tid == 0) a.p16[at] = (int16_t)(need == NEED_NONE ? P_NONE : need + em);
    if (tid < piece) {
        const double t = y * (need == NEED_NONE ? 0.0 : pow2(2 - need)), f = floor(t);
        a.v16[at * piece + tid] = (int16_t)((int)f | (f != t ? 1 : 0));
    }
}

// The same for few blocks: a workgroup joins all heads of a sequence and rounds
// the row itself.  Thread (head, block) finds a weight (SPAN, the most blocks of a
// sequence up to a power of two, times the heads are at most 256), then threads add
// up runs of four neighbouring elements, rows of up to 4096.
constexpr int JOIN_COLS = 4096;
__global__ __launch_bounds__(256) void cache_join_row_kernel(CacheArgs p, AttnArgs a, int span) {
    constexpr int NJ = JOIN_COLS / 1024;
    __shared__ float sw[256];
    __shared__ double sinv[256];
    __shared__ int sem[256], sh[4];
    const int tid = threadIdx.x, seq = blockIdx.x;
    const int len = min(max(p.lengths[seq], 0), p.tokens), nb = (len + 255) >> 8;
    if (tid == 0 && p.lengths[seq] != len) atomicOr(p.flags, IE_FLAG_INDEX);
    const int ex = a.xe[a.x_row ? seq : 0];
    const float r = a.c * pow2f(clip_e(ex));
    // the sums' first blocks are on the way while the weights are found
    const int *num = p.num + (long long)seq * p.blocks * a.cols + 4 * tid;
    v4i x[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        x[j] = v4i{0, 0, 0, 0};
        if (nb > 0 && 4 * tid + 1024 * j < a.cols) x[j] = *(const v4i *)(num + 1024 * j);
    }
    const int head = tid / span, b = tid - head * span;
    float m = -__builtin_inff();
    int n = 0, e = 0;
    if (head < a.heads && b < nb) {
        const int4 t = p.top[((long long)seq * p.blocks + b) * a.heads + head];
        m = __int_as_float(t.x);
        n = t.y;
        e = t.z;
    }
    float top = n ? m : -__builtin_inff();
    int em = n ? max(e, ATT_E_LO) : ATT_E_LO;
    for (int o = 1; o < span; o <<= 1) {  // a head's threads lie in one wave
        top = fmaxf(top, __shfl_xor(top, o, 64));
        em = max(em, __shfl_xor(em, o, 64));
    }
    float w = 0.0f;
    double den = 0.0;
    if (n) {
        const float y = weight(m - top, r);
        den = (double)(y + RINT_MAGIC - RINT_MAGIC) * (double)n;
        w = __builtin_fmaf(y, pow2_down(e - em), RINT_MAGIC) - RINT_MAGIC;
    }
    for (int o = 1; o < span; o <<= 1) den += __shfl_xor(den, o, 64);
    sw[tid] = w;
    if (b == 0) {
        sinv[head] = den > 0.0 ? 1.0 / den : 0.0;
        sem[head] = em;
    }
    __syncthreads();
    double y[NJ][4];
    int need = NEED_NONE;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int c = 4 * tid + 1024 * j, h = c / a.d;
        if (c >= a.cols) break;
        double s[4] = {0, 0, 0, 0};
        for (int i = 0; i < nb; ++i) {
            const v4i v = x[j];
            if (i + 1 < nb) x[j] = *(const v4i *)(num + 1024 * j + (long long)(i + 1) * a.cols);
            const double wt = (double)sw[h * span + i];
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = __builtin_fma(wt, (double)v[k], s[k]);
        }
        MaxMag mx;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[j][k] = s[k] * sinv[h];
        mx.add(y[j][0], y[j][1]);
        mx.add(y[j][2], y[j][3]);
        const int own = need_word(mx.word(), a.q);
        if (own != NEED_NONE) need = max(need, own + sem[h]);
    }
    const int row_e = clamp_exp_flag(max(E_MIN, row_reduce<256>(need, Max{}, sh)), p.flags);
    if (tid == 0) {
        a.ye[seq] = (int8_t)row_e;
        if (ex > ATT_E_HI) atomicOr(p.flags, IE_FLAG_EXP_RANGE);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int c = 4 * tid + 1024 * j;
        if (c >= a.cols) break;
        const double scale = pow2(sem[c / a.d] - row_e);
        int8_t *out = a.y + (long long)seq * a.cols + c;
        int o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __double2loint(__builtin_fma(y[j][k], scale, 6755399441055744.0));  // 1.5 * 2^52
        if (a.out_vec) {
            *(uint32_t *)out = pack4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) out[k] = (int8_t)o[k];
        }
    }
}

hipError_t launch_cache_store(const CacheArgs &c, long long rows, const int8_t *x, const int8_t *xe, int x_row, int width, int first,
                              const int *slots, hipStream_t st) {
    const int nl = c.d <= 16 ? 1 : c.d <= 32 ? 2 : c.d <= 64 ? 4 : 8;
    const long long chunk = rows < STORE_ROWS ? rows : STORE_ROWS, blocks = (chunk * 2 * c.kv + 256 / nl - 1) / (256 / nl);
    const long long chunks = (rows + STORE_ROWS - 1) / STORE_ROWS;
    const dim3 grid((unsigned)(blocks < 8 * NCU ? blocks : 8 * NCU), (unsigned)(chunks < 1024 ? chunks : 1024)), block(256);
    const FastDiv f = make_fastdiv((uint32_t)(2 * c.kv));
    prof_begin(st, PROF_CACHE_STORE);
    if (nl == 1) hipLaunchKernelGGL(cache_store_kernel<1>, grid, block, 0, st, c, rows, x, xe, x_row, width, first, slots, f);
    else if (nl == 2) hipLaunchKernelGGL(cache_store_kernel<2>, grid, block, 0, st, c, rows, x, xe, x_row, width, first, slots, f);
    else if (nl == 4) hipLaunchKernelGGL(cache_store_kernel<4>, grid, block, 0, st, c, rows, x, xe, x_row, width, first, slots, f);
    else hipLaunchKernelGGL(cache_store_kernel<8>, grid, block, 0, st, c, rows, x, xe, x_row, width, first, slots, f);
    prof_end(st, PROF_CACHE_STORE);
    return hipGetLastError();
}

hipError_t launch_cache_attention(const CacheArgs &c, const AttnArgs &a, hipStream_t st) {
    const long long units = (long long)a.kv * ((a.group + 15) / 16), most = (long long)c.n * ((c.blocks + 7) / 8) * 8 * units;
    const long long cap = 4 * NCU;
    const dim3 grid((unsigned)(most < cap ? most : cap));
    prof_begin(st, PROF_ATT_CACHE);
    const int sub = a.group <= 4 ? 4 : a.group <= 8 ? 2 : 1;
#define IE_CASE(DP_, SUB_) \
    if (most && a.d <= DP_ && a.d > DP_ - 64 && sub == SUB_) hipLaunchKernelGGL((cache_attention_kernel<DP_, SUB_>), grid, dim3(256), 0, st, c, a);
    IE_CASE(64, 1) IE_CASE(64, 2) IE_CASE(64, 4) IE_CASE(128, 1) IE_CASE(128, 2) IE_CASE(128, 4)
#undef IE_CASE
    prof_end(st, PROF_ATT_CACHE);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // A workgroup to a sequence where it adds up to eight runs of 1024 sums one after the other (us,
    // that kernel, and joining and rounding with a launch between them: 4 blocks of 8 heads of 64
    // 4.4 and 7; of 32 of 128 9.0 and 8.3, 8 blocks 14 and 8.2)
    int span = 1;
    while (span < c.blocks) span <<= 1;
    if ((a.cols + 1023ll) / 1024 * c.blocks <= 8 && (long long)span * a.heads <= 256 && a.cols <= JOIN_COLS) {
        prof_begin(st, PROF_ATT_JOIN);
        hipLaunchKernelGGL(cache_join_row_kernel, dim3((unsigned)c.n), dim3(256), 0, st, c, a, span);
        prof_end(st, PROF_ATT_JOIN);
        return hipGetLastError();
    }
    // whole heads, or, where these are fewer than two workgroups a CU, 16 elements each (one
    // sequence of 131072 tokens, 32 heads of 128: 9.6 us, whole heads 25; 48 sequences 31 and 8.7)
    AttnArgs r = a;
    const int piece = c.n * a.heads < 2 * NCU ? 16 : a.d;
    r.parts = a.cols / piece;
    r.part = piece;
    prof_begin(st, PROF_ATT_JOIN);
    hipLaunchKernelGGL(cache_join_kernel, dim3((unsigned)(c.n * r.parts)), dim3(256), 0, st, c, r, piece);
    prof_end(st, PROF_ATT_JOIN);
    e = hipGetLastError();
    return e != hipSuccess ? e : launch_attention_round(r, st);
}

}  // namespace ie
