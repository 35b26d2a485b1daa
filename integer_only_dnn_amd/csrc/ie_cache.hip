// Keys and values of 4-bit mantissas in a paged cache, and attention of single
// tokens over it.
//
// A slot of the cache holds, for every key head, head_dim mantissas of 4 bits
// (|C| <= 7) with one exponent for the key and one for the value; two
// mantissas to a byte, the even one in the low half.
#include "ie_attn.h"

#pragma clang fp contract(off)

namespace ie {

constexpr int STORE_ROWS = 4096;  // numbers of a chunk's heads fit 30 bits

// One key or value head of a row: NL lanes with 16 mantissas each.
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
//   o = (sum R(a_b 2^(E_b - E)) N_b) (1 / L) 2^E.
// All sums are exact (below 2^53), so that how blocks are shared out is of no
// account, and each key and value is read once.
//
// A workgroup takes a block of one key head and up to 16 of its query heads,
// a wave 64 of the keys: 16x16x64 products with the keys along the rows and
// the query heads in the columns, so that a lane's 16 weights are 16 bytes of
// the second product's operand.  Values lie in LDS as they come, two elements
// to a byte: a transposing read of 16 columns of bytes is unpacked into two
// operands, the even elements and the odd ones.  Mantissas are unpacked as 16
// times their value (their four bits in a byte's upper half), which the exact
// sums drop.  The next block's keys, values and exponents are in flight while
// one is computed.
template <int DP>  // head size, up: 64 or 128
__global__ __launch_bounds__(256, 4) void cache_attention_kernel(CacheArgs p, AttnArgs a) {
    constexpr int NS = DP / 64, NB = DP / 32, PITCH = DP / 2 + 16, NUM = 20;  // NUM: sums' pitch, one bank to a lane
    __shared__ __align__(16) int8_t sv[256 * PITCH];
    __shared__ __align__(16) float sfk[256], sfv[256];
    __shared__ int scum[256], swave[4], sred[4];
    __shared__ float smax[4][16];
    __shared__ int snum[DP * NUM], ssum[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, c = lane >> 4;
    const int gcs = (a.group + 15) / 16, units = a.kv * gcs, hb = a.d >> 1;
    int s0 = 0, blocks = 0;  // sequences s0 .. s0 + 255 and their blocks of 256 keys
    long long total = 0, before = 0;
    // an item: block b of a sequence, a key head and 16 of its query heads; in
    // groups of eight blocks, a block's heads eight apart: the heads of a slot
    // share cache lines, and these workgroups an XCD
    struct Work {
        long long it;
        int seq, b, kvh, g0, len;
    };
    auto locate = [&](long long it, Work &w) {  // the first item from `it` on that there is
        w.it = it;
        for (; w.it < total; w.it += gridDim.x) {
            const int unit = (int)(w.it / 8 % units), blk = (int)(w.it / 8 / units) * 8 + (int)(w.it % 8);
            if (blk >= blocks) continue;
            int lo = 0, hi = 255;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (scum[mid] > blk) hi = mid;
                else lo = mid + 1;
            }
            w.seq = __builtin_amdgcn_readfirstlane(s0 + lo);
            w.b = __builtin_amdgcn_readfirstlane(blk - (lo ? scum[lo - 1] : 0));
            w.kvh = unit / gcs;
            w.g0 = unit % gcs * 16;
            w.len = min(max(p.lengths[w.seq], 0), p.tokens);
            return true;
        }
        return false;
    };
    // what is read of a block: lane (col, c) takes 16 bytes (DP 64: 8) of the
    // wave's keys col, 16 + col, ..; thread t the exponents of key t
    uint32_t kw[4][2 * NS], vw[4][2 * NS];
    float fk = 0.0f, fv = 0.0f;
    auto slot_of = [&](const Work &w, int j) {
        if (j >= w.len) return -1;
        const int page = p.table[(long long)w.seq * p.per + (j >> p.shift)];
        return page >= 0 && page < p.pages ? (page << p.shift) + (j & (p.page - 1)) : -2;
    };
    auto fetch = [&](const Work &w) {
        const int j0 = 256 * w.b, mine = slot_of(w, j0 + tid);
        int slot[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) slot[t] = slot_of(w, j0 + 64 * wave + 16 * t + col);
        fk = fv = 0.0f;
        if (mine >= 0) {
            const long long at = (long long)mine * p.kv + w.kvh;
            fk = pow2f(clip_e(p.ke[at]));
            fv = pow2f(clip_e(p.ve[at]));
        }
        if (mine == -2) atomicOr(p.flags, IE_FLAG_INDEX);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const long long at = ((long long)slot[t] * p.kv + w.kvh) * hb + 8 * NS * c;
#pragma unroll
            for (int i = 0; i < 2 * NS; ++i) kw[t][i] = vw[t][i] = 0;
            if (slot[t] < 0) continue;
            if (8 * NS * (c + 1) <= hb) {
                __builtin_memcpy(kw[t], p.k + at, 8 * NS);
                __builtin_memcpy(vw[t], p.v + at, 8 * NS);
            } else if (8 * NS * c < hb) {
                __builtin_memcpy(kw[t], p.k + at, 8);
                __builtin_memcpy(vw[t], p.v + at, 8);
            }
        }
    };

    for (s0 = 0; s0 < p.n; s0 += 256) {
        // blocks of the next 256 sequences, and their running sum
        int run = s0 + tid < p.n ? (min(max(p.lengths[s0 + tid], 0), p.tokens) + 255) >> 8 : 0;
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
        __syncthreads();
        blocks = scum[255];
        total = (long long)((blocks + 7) / 8) * 8 * units;
        long long it = (long long)blockIdx.x - before % gridDim.x;
        if (it < 0) it += gridDim.x;
        before += total;
        Work w;
        bool more = locate(it, w);
        if (more) fetch(w);
        while (more) {
            const Work now = w;
            // this block's values and exponents into LDS
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                int8_t *dst = sv + (64 * wave + 16 * t + col) * PITCH + 8 * NS * c;
                __builtin_memcpy(dst, vw[t], 8 * NS);
            }
            sfk[tid] = fk;
            sfv[tid] = fv;
            const int em = wave_max_dpp(__float_as_int(fv));
            if (lane == 0) sred[wave] = em;
            for (int i = tid; i < DP * NUM; i += 256) snum[i] = 0;
            if (tid < 16) ssum[tid] = 0;
            // the query heads, their bytes in the order of unpacked keys
            const int ng = min(16, a.group - now.g0), head = now.kvh * a.group + now.g0 + col;
            const float r = a.c * pow2f(clip_e(a.xe[a.x_row ? now.seq : 0]));
            v4i q[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                q[i] = v4i{0, 0, 0, 0};
                const int e0 = 16 * NS * c + 16 * i;
                if (col < ng && e0 < a.d) {
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
            more = locate(now.it + gridDim.x, w);
            if (more) fetch(w);
            __syncthreads();
            const float fmx = __int_as_float(max(max(sred[0], sred[1]), max(sred[2], sred[3])));
            const int eb = fmx > 0.0f ? (__float_as_int(fmx) >> 23) - 127 : ATT_E_LO;
            const float down = pow2f(-eb);
            float f[4][4], m = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float4 x = *(const float4 *)&sfk[64 * wave + 16 * t + 4 * c];
                const float fs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[t][i] = fs[i] > 0.0f ? (float)acc[t][i] * (0.0625f * fs[i]) : -__builtin_inff();
                    m = fmaxf(m, f[t][i]);
                }
            }
            m = col_max(m);
            if (lane < 16) smax[wave][lane] = m;
            __syncthreads();
            m = fmaxf(fmaxf(smax[0][col], smax[1][col]), fmaxf(smax[2][col], smax[3][col]));
            v4i dh, dl;
            uint32_t sum = 0;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float4 x = *(const float4 *)&sfv[64 * wave + 16 * t + 4 * c];
                const float fvs[4] = {x.x, x.y, x.z, x.w};
                int bits[4];
                uint32_t whole_n[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a key that is not there: a score of minus infinity, whose weight rounds to 0, and a factor of 0
                    const float y = weight(f[t][i] - m, r);
                    bits[i] = __float_as_int(__builtin_fmaf(y, fvs[i] * down, RINT_128));
                    whole_n[i] = (uint32_t)__float_as_int(y + RINT_MAGIC);
                }
                sum += whole_n[0] + whole_n[1];
                sum += whole_n[2] + whole_n[3];
                int h4, l4;
                digits4(bits[0], bits[1], bits[2], bits[3], h4, l4);
                dh[t] = h4;
                dl[t] = l4;
            }
            sum = (uint32_t)col_reduce((int)(sum - 16u * (uint32_t)RINT_BITS), Add{});
            if (lane < ng) atomicAdd(&ssum[lane], (int)sum);
            // the second product: rows are bytes' elements, even ones, then odd ones
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                if (16 * e >= hb) break;
                const int g = lane & 15, kk = g >> 1;
                const int8_t *at = sv + (64 * wave + 16 * (kk >> 2) + 4 * c + (kk & 3)) * PITCH + 16 * e + (g & 1) * 8;
                typedef __attribute__((address_space(3))) v2i lds_v2i;
                const v2i x0 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)at);
                const v2i x1 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(at + 32 * PITCH));
                const uint32_t xs[4] = {(uint32_t)x0.x, (uint32_t)x0.y, (uint32_t)x1.x, (uint32_t)x1.y};
                v4i even, odd;
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    even[z] = (int)(xs[z] << 4 & 0xf0f0f0f0u);
                    odd[z] = (int)(xs[z] & 0xf0f0f0f0u);
                }
                const v4i zero = {0, 0, 0, 0};
                const v4i eh = mfma(even, dh, zero), el = mfma(even, dl, zero), oh = mfma(odd, dh, zero), ol = mfma(odd, dl, zero);
                if (col < ng) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        atomicAdd(&snum[(32 * e + 4 * c + i) * NUM + col], (eh[i] * 256 + el[i]) >> 4);
                        atomicAdd(&snum[(32 * e + 16 + 4 * c + i) * NUM + col], (oh[i] * 256 + ol[i]) >> 4);
                    }
                }
            }
            __syncthreads();
            // this block's sums (elements in their own order)
            const long long out = ((long long)now.seq * p.blocks + now.b) * a.heads + now.kvh * a.group + now.g0;
            for (int i = tid; i < ng * a.d; i += 256) {
                const int hd = i / a.d, e = i - hd * a.d, pos = (e >> 5) * 32 + (e & 1) * 16 + (e >> 1 & 15);
                p.num[out * a.d + i] = snum[pos * NUM + hd];
            }
            if (tid < ng) {
                const float mt = fmaxf(fmaxf(smax[0][tid], smax[1][tid]), fmaxf(smax[2][tid], smax[3][tid]));
                p.top[out + tid] = int4{__float_as_int(mt), ssum[tid], eb, 0};
            }
            __syncthreads();
        }
    }
}

// The blocks of one head of one sequence together, `piece` of its elements to a
// workgroup, as round-to-odd values and a need for a rounding by rows.  Blocks
// are taken 256 at a time: a thread finds the weights of one, then threads of
// four neighbouring elements add up a share of the blocks each.
__global__ __launch_bounds__(256) void cache_join_kernel(CacheArgs p, AttnArgs a, int piece) {
    __shared__ int sh[4];
    __shared__ float sw[256];
    __shared__ double sp[256][4], sden[4];
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
    double s[4] = {0, 0, 0, 0}, den = 0.0;
    for (int b0 = 0; b0 < nb; b0 += 256) {
        const int nc = min(256, nb - b0);
        __syncthreads();
        if (tid < nc) {
            const int4 t = top[(long long)(b0 + tid) * a.heads];
            float w = 0.0f;
            if (t.y) {
                const float x = weight(__int_as_float(t.x) - m, r);
                den += (double)(x + RINT_MAGIC - RINT_MAGIC) * (double)t.y;
                w = __builtin_fmaf(x, pow2f(t.z - em), RINT_MAGIC) - RINT_MAGIC;
            }
            sw[tid] = w;
        }
        __syncthreads();
        if (part < parts) {
#pragma unroll 4
            for (int b = part; b < nc; b += parts) {
                int4 x;
                __builtin_memcpy(&x, num + (long long)(b0 + b) * a.cols + e, 16);
                const double w = (double)sw[b];
                s[0] = __builtin_fma(w, (double)x.x, s[0]);
                s[1] = __builtin_fma(w, (double)x.y, s[1]);
                s[2] = __builtin_fma(w, (double)x.z, s[2]);
                s[3] = __builtin_fma(w, (double)x.w, s[3]);
            }
        }
    }
    // exact sums below 2^53, in any order
#pragma unroll
    for (int k = 0; k < 4; ++k) sp[tid][k] = s[k];
    den = row_reduce<256>(den, Add{}, sden);
    __syncthreads();
    double y = 0.0;
    if (tid < piece) {
        for (int i = 0; i < parts; ++i) y += sp[i * quads + (tid >> 2)][tid & 3];
        y = den > 0.0 ? y * (1.0 / den) : 0.0;
    }
    const int need = need_word(row_reduce<256>(__double2hiint(y) & 0x7fffffff, Max{}, sh), a.q);
    const long long at = (long long)seq * a.heads * pieces + part_of;
    if (tid == 0) a.p16[at] = (int16_t)(need == NEED_NONE ? P_NONE : need + em);
    if (tid < piece) {
        const double t = y * (need == NEED_NONE ? 0.0 : pow2(2 - need)), f = floor(t);
        a.v16[at * piece + tid] = (int16_t)((int)f | (f != t ? 1 : 0));
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
    if (a.d <= 64) hipLaunchKernelGGL(cache_attention_kernel<64>, grid, dim3(256), 0, st, c, a);
    else hipLaunchKernelGGL(cache_attention_kernel<128>, grid, dim3(256), 0, st, c, a);
    prof_end(st, PROF_ATT_CACHE);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // whole heads, or, where these are too few workgroups, 16 elements each
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
