// Keys and values of 4-bit mantissas in a paged cache, and attention of single
// tokens over it.
//
// A slot of the cache holds, for every key head, head_dim mantissas of 4 bits
// (|C| <= 7) with one exponent for the key and one for the value; two
// mantissas to a byte, the even one in the low half.
#include "ie_attn.h"

#pragma clang fp contract(off)

namespace ie {

typedef int v4acc __attribute__((ext_vector_type(4)));

// One key or value head of a row: 16 lanes with eight mantissas each.
__global__ __launch_bounds__(256) void cache_store_kernel(CacheArgs p, long long rows, const int8_t *x, const int8_t *xe, int x_row,
                                                          int width, int first, const int *slots) {
    const int parts = 2 * p.kv, lane = threadIdx.x & 15;
    const long long total = rows * parts, slot_max = (long long)p.pages * p.page;
    for (long long i = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); i < (total + 15) / 16 * 16; i += (long long)gridDim.x * 16) {
        const bool in = i < total;
        const long long row = in ? i / parts : 0;
        const int part = in ? (int)(i - row * parts) : 0;
        const long long slot = in ? slots[row] : -1;
        if (slot >= slot_max && lane == 0) atomicOr(p.flags, IE_FLAG_INDEX);
        const bool on = slot >= 0 && slot < slot_max;
        const int8_t *src = x + row * width + first + part * p.d + 8 * lane;
        uint32_t w[2] = {0, 0};
        if (on && 8 * lane < p.d) __builtin_memcpy(w, src, 8);
        int m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max(m, abs(byte_of(w[k >> 2], k & 3)));
        m = lane_reduce<16>(m, Max{});
        const int ex = on ? (int)xe[x_row ? row : 0] : 0;
        int e = max(E_MIN, need32(m, ex, 3));
        const int s = e - ex;
        uint32_t o = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) o |= (uint32_t)(rne_shift32(byte_of(w[k >> 2], k & 3), s) & 15) << (4 * k);
        if (!on) continue;
        const bool val = part >= p.kv;
        const long long at = slot * p.kv + (val ? part - p.kv : part);
        if (lane == 0) (val ? p.ve : p.ke)[at] = (int8_t)clamp_exp_flag(e, p.flags);
        if (8 * lane < p.d) *(uint32_t *)((val ? p.v : p.k) + at * (p.d >> 1) + 4 * lane) = o;
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
// the second product's operand.  Mantissas are unpacked as 16 times their
// value (their four bits in a byte's upper half), which the exact sums drop.
template <int DP>  // head size, up: 64 or 128
__global__ __launch_bounds__(256) void cache_attention_kernel(CacheArgs p, AttnArgs a) {
    constexpr int NS = DP / 64, PITCH = DP + 16;
    __shared__ __align__(16) int8_t sv[256 * PITCH];
    __shared__ __align__(16) float sfk[256], sfv[256];
    __shared__ int sslot[256], scum[256], swave[4], sred[4];
    __shared__ float smax[4][16];
    __shared__ int snum[16 * DP], ssum[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, c = lane >> 4;
    const int gcs = (a.group + 15) / 16, units = a.kv * gcs;
    if (blockIdx.x == 0)
        for (int i = tid; i < p.n; i += 256) p.count[i] = 0;
    long long before = 0;  // items of the sequences of earlier chunks
    for (int s0 = 0; s0 < p.n; s0 += 256) {
        // blocks of 256 keys of the next 256 sequences, and their running sum
        int nb = 0;
        if (s0 + tid < p.n) nb = (min(max(p.lengths[s0 + tid], 0), p.tokens) + 255) >> 8;
        int run = nb;
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
        const int blocks = scum[255];
        // items in groups of eight blocks, a block's heads eight apart: the
        // heads of a slot share cache lines, and these workgroups an XCD
        const long long total = (long long)((blocks + 7) / 8) * 8 * units;
        long long it = (long long)blockIdx.x - before % gridDim.x;
        if (it < 0) it += gridDim.x;
        before += total;
        for (; it < total; it += gridDim.x) {
            const int unit = (int)(it / 8 % units), blk = (int)(it / 8 / units) * 8 + (int)(it % 8);
            if (blk >= blocks) continue;
            int lo = 0, hi = 255;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (scum[mid] > blk) hi = mid;
                else lo = mid + 1;
            }
            const int seq = s0 + lo, b = blk - (lo ? scum[lo - 1] : 0);
            const int kvh = unit / gcs, g0 = unit % gcs * 16, ng = min(16, a.group - g0);
            const int len = min(max(p.lengths[seq], 0), p.tokens);
            // slots and exponents of the block's keys
            const int j = 256 * b + tid;
            int slot = -1;
            float fv = 0.0f;
            if (j < len) {
                const int page = p.table[(long long)seq * p.per + (j >> p.shift)];
                if (page >= 0 && page < p.pages) {
                    slot = (page << p.shift) + (j & (p.page - 1));
                    const long long at = (long long)slot * p.kv + kvh;
                    sfk[tid] = pow2f(clip_e(p.ke[at]));
                    fv = pow2f(clip_e(p.ve[at]));
                } else {
                    atomicOr(p.flags, IE_FLAG_INDEX);
                }
            }
            if (slot < 0) sfk[tid] = 0.0f;
            sfv[tid] = fv;
            sslot[tid] = slot;
            const int em = wave_max_dpp(__float_as_int(fv));
            if (lane == 0) sred[wave] = em;
            for (int i = tid; i < 16 * DP; i += 256) snum[i] = 0;
            if (tid < 16) ssum[tid] = 0;
            __syncthreads();
            const float fmx = __int_as_float(max(max(sred[0], sred[1]), max(sred[2], sred[3])));
            const int eb = fmx > 0.0f ? (__float_as_int(fmx) >> 23) - 127 : ATT_E_LO;
            const float down = pow2f(-eb);
            // keys and values of this wave's 64 slots: lane (col, c) takes 16
            // bytes (DP 64: 8) of keys col, 16 + col, ...
            uint32_t kw[4][2 * NS], vw[4][2 * NS];
            const int hb = a.d >> 1;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int s = sslot[64 * wave + 16 * t + col];
                const long long at = ((long long)s * p.kv + kvh) * hb + 8 * NS * c;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    uint2 k2 = {0, 0}, v2 = {0, 0};
                    if (s >= 0 && 8 * NS * c + 8 * i < hb) {
                        k2 = *(const uint2 *)(p.k + at + 8 * i);
                        v2 = *(const uint2 *)(p.v + at + 8 * i);
                    }
                    kw[t][2 * i] = k2.x;
                    kw[t][2 * i + 1] = k2.y;
                    vw[t][2 * i] = v2.x;
                    vw[t][2 * i + 1] = v2.y;
                }
            }
            // the query heads, their bytes in the order of unpacked keys
            const int head = kvh * a.group + g0 + col;
            const int eq = clip_e(a.xe[a.x_row ? seq : 0]);
            const float r = a.c * pow2f(eq);
            v4i q[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                q[i] = v4i{0, 0, 0, 0};
                const int e0 = 16 * NS * c + 16 * i;
                if (col < ng && e0 < a.d) {
                    uint32_t w[4];
                    __builtin_memcpy(w, a.x + (long long)seq * a.width + (long long)head * a.d + e0, 16);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        q[i][2 * z] = (int)__builtin_amdgcn_perm(w[2 * z + 1], w[2 * z], 0x06040200u);
                        q[i][2 * z + 1] = (int)__builtin_amdgcn_perm(w[2 * z + 1], w[2 * z], 0x07050301u);
                    }
                }
            }
            v4acc acc[4];
            float m = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                acc[t] = v4acc{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    v4i k;
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        k[2 * z] = (int)(kw[t][2 * i + z] << 4 & 0xf0f0f0f0u);
                        k[2 * z + 1] = (int)(kw[t][2 * i + z] & 0xf0f0f0f0u);
                    }
                    acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(k, q[i], acc[t], 0, 0, 0);
                }
            }
            float f[4][4], score[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float4 fk = *(const float4 *)&sfk[64 * wave + 16 * t + 4 * c];
                const float fs[4] = {fk.x, fk.y, fk.z, fk.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[t][i] = fs[i];
                    score[t][i] = (float)acc[t][i] * (0.0625f * fs[i]);
                    m = fmaxf(m, fs[i] > 0.0f ? score[t][i] : -__builtin_inff());
                }
            }
            m = col_max(m);
            if (lane < 16) smax[wave][lane] = m;
            // values, unpacked
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                int8_t *dst = sv + (64 * wave + 16 * t + col) * PITCH + 16 * NS * c;
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    *(v4i *)(dst + 16 * i) = v4i{(int)(vw[t][2 * i] << 4 & 0xf0f0f0f0u), (int)(vw[t][2 * i] & 0xf0f0f0f0u),
                                                 (int)(vw[t][2 * i + 1] << 4 & 0xf0f0f0f0u), (int)(vw[t][2 * i + 1] & 0xf0f0f0f0u)};
            }
            __syncthreads();
            m = fmaxf(fmaxf(smax[0][col], smax[1][col]), fmaxf(smax[2][col], smax[3][col]));
            v4i dh, dl;
            uint32_t sum = 0;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float4 f4 = *(const float4 *)&sfv[64 * wave + 16 * t + 4 * c];
                const float fvs[4] = {f4.x, f4.y, f4.z, f4.w};
                int bits[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float w = weight(score[t][i] - m, r);
                    if (!(f[t][i] > 0.0f)) w = 0.0f;
                    bits[i] = __float_as_int(__builtin_fmaf(w, fvs[i] * down, RINT_128));
                    sum += (uint32_t)__float_as_int(w + RINT_MAGIC) - (uint32_t)RINT_BITS;
                }
                int h4, l4;
                digits4(bits[0], bits[1], bits[2], bits[3], h4, l4);
                dh[t] = h4;
                dl[t] = l4;
            }
            sum = (uint32_t)swap_reduce<16>((int)sum, Add{});
            sum = (uint32_t)swap_reduce<32>((int)sum, Add{});
            if (lane < 16) atomicAdd(&ssum[lane], (int)sum);
            // the second product: rows are the values' elements as unpacked
#pragma unroll
            for (int dt = 0; dt < DP / 16; ++dt) {
                const int g = lane & 15, kk = g >> 1;
                const int8_t *at = sv + (64 * wave + 16 * (kk >> 2) + 4 * c + (kk & 3)) * PITCH + 16 * dt + (g & 1) * 8;
                typedef __attribute__((address_space(3))) v2i lds_v2i;
                const v2i x0 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)at);
                const v2i x1 = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(at + 32 * PITCH));
                const v4i vt = {x0.x, x0.y, x1.x, x1.y};
                v4acc ah = {0, 0, 0, 0}, al = {0, 0, 0, 0};
                ah = __builtin_amdgcn_mfma_i32_16x16x64_i8(vt, dh, ah, 0, 0, 0);
                al = __builtin_amdgcn_mfma_i32_16x16x64_i8(vt, dl, al, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) atomicAdd(&snum[col * DP + 16 * dt + 4 * c + i], (ah[i] * 256 + al[i]) >> 4);
            }
            __syncthreads();
            // this block's sums (elements in their own order)
            const long long out = ((long long)seq * p.blocks + b) * a.heads + kvh * a.group + g0;
            for (int i = tid; i < ng * a.d; i += 256) {
                const int hd = i / a.d, e = i - hd * a.d, pos = (e & ~7) + (e >> 1 & 3) + (e & 1) * 4;
                p.num[out * a.d + i] = snum[hd * DP + pos];
            }
            if (tid < ng) {
                const float mt = fmaxf(fmaxf(smax[0][tid], smax[1][tid]), fmaxf(smax[2][tid], smax[3][tid]));
                p.top[out + tid] = int4{__float_as_int(mt), ssum[tid], eb, 0};
            }
            __syncthreads();
        }
    }
}

// The blocks of one head of one sequence together, then, by the workgroup that
// finishes a sequence, its heads rounded into one exponent.
__global__ __launch_bounds__(256) void cache_join_kernel(CacheArgs p, AttnArgs a) {
    __shared__ double sden[4];
    __shared__ float sm[4];
    __shared__ int sh[4];
    __shared__ int slast;
    const int seq = blockIdx.x / a.heads, head = blockIdx.x - seq * a.heads, tid = threadIdx.x;
    const int len = min(max(p.lengths[seq], 0), p.tokens), nb = (len + 255) >> 8;
    if (tid == 0 && p.lengths[seq] != len) atomicOr(p.flags, IE_FLAG_INDEX);
    const int4 *top = p.top + (long long)seq * p.blocks * a.heads + head;
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
    // elements in the lanes, blocks shared by the two halves of the workgroup
    // or its quarters (head sizes of up to 64)
    const int lanes = a.d <= 64 ? 64 : 128, part = tid / lanes, parts = 256 / lanes, e = tid % lanes;
    const int *num = p.num + ((long long)seq * p.blocks * a.heads + head) * a.d;
    double s = 0.0, den = 0.0;
    for (int b = part; b < nb; b += parts) {
        const int4 t = top[(long long)b * a.heads];
        if (!t.y) continue;
        const float w = weight(__int_as_float(t.x) - m, r);
        den += (double)(w + RINT_MAGIC - RINT_MAGIC) * (double)t.y;
        const float wv = __builtin_fmaf(w, pow2f(t.z - em), RINT_MAGIC) - RINT_MAGIC;
        if (e < a.d) s += (double)wv * (double)num[(long long)b * a.heads * a.d + e];
    }
    __shared__ double sp[256];
    sp[tid] = s;
    if (e == 0) sden[part] = den;
    __syncthreads();
    double y = 0.0, total = 0.0;
    for (int i = 0; i < parts; ++i) {
        total += sden[i];
        if (tid < lanes) y += sp[i * lanes + tid];
    }
    y = tid < a.d && total > 0.0 ? y * (1.0 / total) : 0.0;
    const int word = __double2hiint(y) & 0x7fffffff;
    const int need = need_word(row_reduce<256>(word, Max{}, sh), a.q);
    const long long at = (long long)seq * a.heads + head;
    if (tid == 0) a.p16[at] = (int16_t)(need == NEED_NONE ? P_NONE : need + em);
    if (tid < a.d) {
        const double t = y * (need == NEED_NONE ? 0.0 : pow2(2 - need)), f = floor(t);
        a.v16[at * a.d + tid] = (int16_t)((int)f | (f != t ? 1 : 0));
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) slast = atomicAdd(&p.count[seq], 1) == a.heads - 1;
    __syncthreads();
    if (!slast) return;
    __threadfence();
    const volatile int16_t *needs = a.p16 + (long long)seq * a.heads;
    int ne = P_NONE;
    for (int i = tid; i < a.heads; i += 256) ne = max(ne, (int)needs[i]);
    ne = row_reduce<256>(ne, Max{}, sh);
    const int ey = clamp_exp_flag(max(E_MIN, ne), a.flags);
    if (tid == 0) {
        a.ye[seq] = (int8_t)ey;
        if (a.xe[a.x_row ? seq : 0] > ATT_E_HI) atomicOr(a.flags, IE_FLAG_EXP_RANGE);
    }
    const volatile int16_t *v = a.v16 + (long long)seq * a.cols;
    for (int i = tid; i < a.cols; i += 256)
        a.y[(long long)seq * a.cols + i] = (int8_t)rne_shift32((int)v[i], ey - ((int)needs[i / a.d] - 2));
}

hipError_t launch_cache_store(const CacheArgs &c, long long rows, const int8_t *x, const int8_t *xe, int x_row, int width, int first,
                              const int *slots, hipStream_t st) {
    const long long blocks = (rows * 2 * c.kv + 15) / 16;
    prof_begin(st, PROF_CACHE_STORE);
    hipLaunchKernelGGL(cache_store_kernel, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, st, c, rows, x, xe, x_row,
                       width, first, slots);
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
    prof_begin(st, PROF_ATT_JOIN);
    hipLaunchKernelGGL(cache_join_kernel, dim3((unsigned)(c.n * a.heads)), dim3(256), 0, st, c, a);
    prof_end(st, PROF_ATT_JOIN);
    return hipGetLastError();
}

}  // namespace ie
