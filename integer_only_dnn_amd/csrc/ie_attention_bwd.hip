// Softmax attention over packed sequences, backward.
//
// With the forward pass's weights w_ij, sums L_i and results O (as rounded),
// p_ij = w_ij / L_i:
//   u_ij = dP_ij - D_i,  dP_ij = (dO_i . v_j) 2^(e_j),  D_i = (dO_i . O_i) 2^(eO_i),
// exact products, the difference rounded to fp32, in units of 2^(eo_i) (eo the
// exponents of dO);
//   dQ_i = scale sum_j p_ij u_ij k_j,  dK_j = scale sum_i p_ij u_ij q_i,
//   dV_j = sum_i p_ij dO_i.
// The sums run over integers, so that their order is of no account:
//   dQ: B = R(s 2^(e_j - sigma_i)), s = w u rounded to fp32;
//   dV: A = R((w a_i) 2^(-kappa_j)), a_i = 2^(max(eo_i - max eo, -60)) / L_i in fp32;
//   dK: C = R((s b_i) 2^(6 - lambda_j)), b_i = a_i 2^(e_i) in units of 2^(max lambda).
// sigma, kappa, lambda are powers of two that bound what they scale (|dO_i . v_j|
// by the product of the norms), taken over the rows that meet in the sum, so
// |A|, |B| <= 32512 and |C| <= 64 * 32512: two and three int8 digits.  C has
// three, as it sums rows whose sizes differ most: with two, the bounds left it
// a root mean square of four units.
#include "ie_attn.h"

#pragma clang fp contract(off)

namespace ie {

__device__ __forceinline__ int bits_of(uint32_t n) { return 32 - __clz((int)n); }  // n = 0: 0

// A row's products of dO with O and itself by head, and the norms of its
// values: 16 lanes a head, eight elements each.
__global__ __launch_bounds__(256) void attn_dot_kernel(AttnArgs p, AttnBwd b) {
    const int lane = threadIdx.x & 15, parts = p.heads + p.kv;
    const long long total = p.rows * parts;
    for (long long i = (long long)blockIdx.x * 16 + (threadIdx.x >> 4); i < (total + 15) / 16 * 16; i += (long long)gridDim.x * 16) {
        const long long row = i < total ? i / parts : 0;
        const int part = i < total ? (int)(i - row * parts) : 0;
        uint32_t x[2] = {0, 0}, y[2] = {0, 0};
        if (part < p.heads) {
            load_run<8>(b.dy + row * p.heads * p.d + part * p.d, 8 * lane, p.d, x);
            load_run<8>(b.o + row * p.heads * p.d + part * p.d, 8 * lane, p.d, y);
        } else {
            load_run<8>(p.x + row * p.width + (part + p.kv) * p.d, 8 * lane, p.d, x);
        }
        int dot = 0, sq = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            dot = __builtin_amdgcn_sdot4((int)x[k], (int)y[k], dot, false);
            sq = __builtin_amdgcn_sdot4((int)x[k], (int)x[k], sq, false);
        }
        dot = lane_reduce<16>(dot, Add{});
        sq = lane_reduce<16>(sq, Add{});
        if (lane || i >= total) continue;
        const int size = (bits_of((uint32_t)sq) + 1) >> 1;  // |.| < 2^size
        if (part < p.heads) b.dots[row * p.heads + part] = int2{dot, size};
        else b.norm[row * p.kv + part - p.heads] = (int8_t)size;
    }
}

// The scales of one sequence and key head: a workgroup each.  Suffix maxima
// (causal: a key meets the queries from its own on) by runs of a thread.
__global__ __launch_bounds__(256) void attn_scale_kernel(AttnArgs p, AttnBwd b) {
    __shared__ int sh[4];
    __shared__ int ska[256], skl[256];
    const int seq = blockIdx.x / p.kv, kvh = blockIdx.x - seq * p.kv, tid = threadIdx.x;
    const Span sp = seq_span(p, seq);
    if (sp.n <= 0) return;
    int e_top = ATT_E_LO, n_top = -4096, r_top = -4096, o_top = E_MIN;
    for (int t = tid; t < sp.n; t += 256) {
        const long long row = sp.a + t;
        const int e = clip_e(p.xe[p.x_row ? row : 0]), nu = b.norm[row * p.kv + kvh] + e;
        e_top = max(e_top, e);
        n_top = max(n_top, nu);
        r_top = max(r_top, nu + e);
        o_top = max(o_top, (int)b.dye[b.dy_row ? row : 0]);
    }
    e_top = row_reduce<256>(e_top, Max{}, sh);
    n_top = row_reduce<256>(n_top, Max{}, sh);
    r_top = row_reduce<256>(r_top, Max{}, sh);
    o_top = row_reduce<256>(o_top, Max{}, sh);
    // alpha and lambda of a query: a_i < 2^alpha, a_i |u| 2^(e_i) < 2^lambda
    auto query = [&](int t, int g, int &alpha, int &lam, float &a, float &dot, int &rise) {
        const long long row = sp.a + t;
        const int h = kvh * p.group + g, e = clip_e(p.xe[p.x_row ? row : 0]);
        const int2 d = b.dots[row * p.heads + h];
        const int eo = clip_e(b.oe[row]), delta = bits_of((uint32_t)abs(d.x)) + eo;
        const uint32_t sum = (uint32_t)p.stats[row * p.heads + h].y;
        a = (float)(1.0 / (double)sum) * pow2f(max((int)b.dye[b.dy_row ? row : 0] - o_top, -60));
        alpha = (__float_as_int(a) >> 23) - 126;
        lam = alpha + e + max(d.y + n_top, delta) + 1;
        dot = (float)d.x * pow2f(eo);
        rise = max(d.y + r_top, delta + e_top) + 1;
    };
    const int per = (sp.n + 255) / 256, t0 = min(tid * per, sp.n), t1 = min(t0 + per, sp.n);
    int ka = -4096, kl = -4096;
    for (int t = t0; t < t1; ++t)
        for (int g = 0; g < p.group; ++g) {
            int alpha, lam, rise;
            float a, dot;
            query(t, g, alpha, lam, a, dot, rise);
            ka = max(ka, alpha);
            kl = max(kl, lam);
        }
    ska[tid] = ka;
    skl[tid] = kl;
    __syncthreads();
    int later_a = -4096, later_l = -4096, all_a = -4096, whole = -4096;
    for (int i = 0; i < 256; ++i) {
        all_a = max(all_a, ska[i]);
        whole = max(whole, skl[i]);
        if (i > tid) {
            later_a = max(later_a, ska[i]);
            later_l = max(later_l, skl[i]);
        }
    }
    for (int t = t1 - 1; t >= t0; --t) {
        const long long row = sp.a + t;
        const int e = clip_e(p.xe[p.x_row ? row : 0]), ed = b.dye[b.dy_row ? row : 0];
        for (int g = 0; g < p.group; ++g) {
            int alpha, lam, rise;
            float a, dot;
            query(t, g, alpha, lam, a, dot, rise);
            later_a = max(later_a, alpha);
            later_l = max(later_l, lam);
            const int h = kvh * p.group + g;
            const int2 st = p.stats[row * p.heads + h];
            AttnRow q;
            q.m = __int_as_float(st.x);
            q.r = p.c * pow2f(e);
            q.dot = dot;
            q.a = a;
            q.b = (float)((double)a * pow2(e - whole));
            q.s = pow2f(max(-rise, -126));
            q.e = rise + ed;
            q.sum = (uint32_t)st.y;
            b.row[(long long)h * p.rows + row] = q;
        }
        AttnKey k;
        k.kappa = p.causal ? later_a : all_a;
        k.lambda = max((p.causal ? later_l : whole) - whole, -96);
        k.ev = k.kappa + o_top;
        k.ek = k.lambda - 6 + whole + o_top;
        b.key[(long long)kvh * p.rows + row] = k;
    }
}

// dQ: a workgroup of four waves takes 128 queries of a head, one to a lane
// pair, as in the forward pass; keys and values pass through LDS.
template <int DP, bool ROW, bool CAUSAL>
__global__ __launch_bounds__(256) void attn_dq_kernel(AttnArgs p, AttnBwd bw, int slots) {
    using T = HeadTile<DP>;
    constexpr int NS = DP / 32;
    __shared__ __align__(16) int8_t sk[2][T::BYTES], sv[2][T::BYTES];
    __shared__ __align__(16) float sf[2][64];
    const long long item = xcd_item((long long)slots * p.heads);
    if (item < 0) return;
    const int gh = (int)(item % p.group), rest = (int)(item / p.group);
    const int kvh = rest / slots, slot = CAUSAL ? slots - 1 - rest % slots : rest % slots;
    const int h = kvh * p.group + gh;
    int q0, seq;
    const Span sp = slot_span(p, slot, 128, q0, seq);
    if (q0 >= sp.n) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
    const int n = sp.n, qw = q0 + 32 * wave, qi = qw + (lane & 31);
    const bool ok = qi < n;
    const int8_t *base = p.x + (long long)sp.a * p.width;
    const int8_t *kh = base + (p.heads + kvh) * p.d, *vh = kh + (long long)p.kv * p.d;
    const int8_t *xe = p.xe + (ROW ? sp.a : 0);
    const long long row = sp.a + qi;
    v4i q[NS], g[NS];
    head_regs<DP>(base + (long long)qi * p.width + h * p.d, ok, p.d, p.vec, lane, q);
    head_regs<DP>(bw.dy + row * p.heads * p.d + h * p.d, ok, p.d, bw.dy_vec, lane, g);
    const AttnRow st = bw.row[(long long)h * p.rows + sp.a + min(qi, n - 1)];
    const float fe0 = pow2f(clip_e(xe[0]));
    const int keys = CAUSAL ? min(n, q0 + 128) : n, tiles = (keys + 63) / 64;
    const int last = CAUSAL ? min(n, qw + 32) : n;
    const bool idle = qw >= n;
    T k, v;
    float fe = 0.0f;
    auto fetch = [&](int t) {
        k.fetch(kh, p.width, 64 * t, keys, p.d, p.vec);
        v.fetch(vh, p.width, 64 * t, keys, p.d, p.vec);
        if (ROW && tid < 64) fe = pow2f(clip_e(xe[min(64 * t + tid, n - 1)]));
    };
    v16i hi[NS] = {}, lo[NS] = {};
    fetch(0);
    for (int t = 0; t < tiles; ++t) {
        k.put(sk[t & 1]);
        v.put(sv[t & 1]);
        if (ROW && tid < 64) sf[t & 1][tid] = fe;
        if (t + 1 < tiles) fetch(t + 1);
        __syncthreads();
#pragma unroll
        for (int b = 0; b < 64; b += 32) {
            const int j0 = 64 * t + b;
            if (idle || j0 >= last) continue;
            v16i s = {}, dp = {};
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                s = mfma(T::frag_r(sk[t & 1], b, i, lane), q[i], s);
                dp = mfma(T::frag_r(sv[t & 1], b, i, lane), g[i], dp);
            }
            const bool all = j0 + 32 <= (CAUSAL ? qw + 1 : n);
            v4i dh, dl;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 f = ROW ? *(const float4 *)&sf[t & 1][b + 8 * c + 4 * half] : float4{fe0, fe0, fe0, fe0};
                const float fs[4] = {f.x, f.y, f.z, f.w};
                int bits[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + 8 * c + 4 * half + i;
                    float w = weight(__builtin_fmaf((float)s[4 * c + i], fs[i], -st.m), st.r);
                    if (!all && !(CAUSAL ? j <= qi : j < n)) w = 0.0f;
                    const float u = __builtin_fmaf((float)dp[4 * c + i], fs[i], -st.dot);
                    bits[i] = __float_as_int(__builtin_fmaf(w * u * fs[i], st.s, RINT_128));
                }
                int x, y;
                digits4(bits[0], bits[1], bits[2], bits[3], x, y);
                dh[c] = x;
                dl[c] = y;
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const v4i kt = T::frag_t(sk[t & 1], b, i, lane);
                hi[i] = mfma(kt, dh, hi[i]);
                lo[i] = mfma(kt, dl, lo[i]);
            }
        }
    }
    if (idle) return;
    const double rate = p.scale / (double)st.sum;
    double y[16 * NS];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 16; ++i) y[16 * s + i] = __builtin_fma((double)hi[s][i], 256.0, (double)lo[s][i]) * rate;
    store_odd(y, st.e, p.q, ok, p.d, lane, p.v16 + row * p.cols + h * p.d, p.p16 + row * p.parts + h);
}

// dK and dV: a workgroup of four waves takes 128 keys, one to a lane pair, and
// runs over the query heads that share them and their queries.
template <int DP, bool CAUSAL>
__global__ __launch_bounds__(256) void attn_dkv_kernel(AttnArgs p, AttnBwd bw, int slots) {
    using T = HeadTile<DP>;
    constexpr int NS = DP / 32;
    __shared__ __align__(16) int8_t sq[2][T::BYTES], sg[2][T::BYTES];
    __shared__ __align__(16) float sr[2][5][64];
    const long long item = xcd_item((long long)slots * p.kv);
    if (item < 0) return;
    const int kvh = (int)(item / slots), slot = (int)(item % slots);
    int k0, seq;
    const Span sp = slot_span(p, slot, 128, k0, seq);
    if (k0 >= sp.n) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
    const int n = sp.n, kw = k0 + 32 * wave, kj = kw + (lane & 31);
    const bool ok = kj < n, idle = kw >= n;
    const int8_t *base = p.x + (long long)sp.a * p.width;
    const long long row = sp.a + kj;
    v4i k[NS], v[NS];
    head_regs<DP>(base + (long long)kj * p.width + (p.heads + kvh) * p.d, ok, p.d, p.vec, lane, k);
    head_regs<DP>(base + (long long)kj * p.width + (p.heads + p.kv + kvh) * p.d, ok, p.d, p.vec, lane, v);
    const AttnKey key = bw.key[(long long)kvh * p.rows + sp.a + min(kj, n - 1)];
    const float f = pow2f(clip_e(p.xe[p.x_row ? sp.a + min(kj, n - 1) : 0]));
    const float sv = pow2f(min(-key.kappa, 126)), sk = pow2f(min(6 - key.lambda, 126));
    const int first = CAUSAL ? k0 / 64 : 0, tiles = (n + 63) / 64 - first, steps = tiles * p.group;
    T q, g;
    AttnRow rec;
    auto fetch = [&](int i) {
        const int h = kvh * p.group + i / tiles, t = first + i % tiles;
        q.fetch(base + h * p.d, p.width, 64 * t, n, p.d, p.vec);
        g.fetch(bw.dy + (long long)sp.a * p.heads * p.d + h * p.d, (long long)p.heads * p.d, 64 * t, n, p.d, bw.dy_vec);
        if (tid < 64) rec = bw.row[(long long)h * p.rows + sp.a + min(64 * t + tid, n - 1)];
    };
    v16i vh[NS] = {}, vl[NS] = {}, c2[NS] = {}, c1[NS] = {}, c0[NS] = {};
    const v4i bias = {(int)0xc0c0c0c0u, (int)0xc0c0c0c0u, (int)0xc0c0c0c0u, (int)0xc0c0c0c0u};  // -64
    fetch(0);
    for (int i = 0; i < steps; ++i) {
        const int buf = i & 1, t = first + i % tiles;
        q.put(sq[buf]);
        g.put(sg[buf]);
        if (tid < 64) {
            sr[buf][0][tid] = rec.m;
            sr[buf][1][tid] = rec.r;
            sr[buf][2][tid] = rec.dot;
            sr[buf][3][tid] = rec.a;
            sr[buf][4][tid] = rec.b;
        }
        if (i + 1 < steps) fetch(i + 1);
        __syncthreads();
#pragma unroll
        for (int b = 0; b < 64; b += 32) {
            const int i0 = 64 * t + b;
            if (idle || i0 >= n || (CAUSAL && i0 + 31 < kw)) continue;
            v16i s = {}, dp = {};
#pragma unroll
            for (int z = 0; z < NS; ++z) {
                s = mfma(T::frag_r(sq[buf], b, z, lane), k[z], s);
                dp = mfma(T::frag_r(sg[buf], b, z, lane), v[z], dp);
            }
            const bool all = i0 + 32 <= n && (!CAUSAL || kw + 31 <= i0);
            v4i ah, al, d2, d1, d0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float r5[5][4];
#pragma unroll
                for (int z = 0; z < 5; ++z) {
                    const float4 x = *(const float4 *)&sr[buf][z][b + 8 * c + 4 * half];
                    r5[z][0] = x.x;
                    r5[z][1] = x.y;
                    r5[z][2] = x.z;
                    r5[z][3] = x.w;
                }
                int ab[4], cb[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int qi = i0 + 8 * c + 4 * half + x;
                    float w = weight(__builtin_fmaf((float)s[4 * c + x], f, -r5[0][x]), r5[1][x]);
                    if (!all && !(qi < n && (!CAUSAL || kj <= qi))) w = 0.0f;
                    const float u = __builtin_fmaf((float)dp[4 * c + x], f, -r5[2][x]);
                    ab[x] = __float_as_int(__builtin_fmaf(w * r5[3][x], sv, RINT_128));
                    cb[x] = __float_as_int(__builtin_fmaf(w * u * r5[4][x], sk, RINT_MAGIC + 32896.0f));
                }
                int x, y, z;
                digits4(ab[0], ab[1], ab[2], ab[3], x, y);
                ah[c] = x;
                al[c] = y;
                digits3x4(cb[0], cb[1], cb[2], cb[3], x, y, z);
                d2[c] = x;
                d1[c] = y;
                d0[c] = z;
            }
#pragma unroll
            for (int z = 0; z < NS; ++z) {
                const v4i gt = T::frag_t(sg[buf], b, z, lane), qt = T::frag_t(sq[buf], b, z, lane);
                vh[z] = mfma(gt, ah, vh[z]);
                vl[z] = mfma(gt, al, vl[z]);
                c2[z] = mfma(qt, bias, c2[z]);
                c2[z] = mfma(qt, d2, c2[z]);
                c1[z] = mfma(qt, d1, c1[z]);
                c0[z] = mfma(qt, d0, c0[z]);
            }
        }
    }
    if (idle) return;
    double y[16 * NS];
    int16_t *out = p.v16 + row * p.cols, *need = p.p16 + row * p.parts;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            y[16 * s + i] = ((double)c2[s][i] * 65536.0 + ((double)c1[s][i] * 256.0 + (double)c0[s][i])) * p.scale;
    store_odd(y, key.ek, p.q, ok, p.d, lane, out + (p.heads + kvh) * p.d, need + p.heads + kvh);
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 16; ++i) y[16 * s + i] = (double)vh[s][i] * 256.0 + (double)vl[s][i];
    store_odd(y, key.ev, p.q, ok, p.d, lane, out + (p.heads + p.kv + kvh) * p.d, need + p.heads + p.kv + kvh);
}

template <int DP>
static void dq(const AttnArgs &a, const AttnBwd &b, int slots, dim3 grid, hipStream_t st) {
    const dim3 block(256);
    if (a.x_row) {
        if (a.causal) hipLaunchKernelGGL((attn_dq_kernel<DP, true, true>), grid, block, 0, st, a, b, slots);
        else hipLaunchKernelGGL((attn_dq_kernel<DP, true, false>), grid, block, 0, st, a, b, slots);
    } else {
        if (a.causal) hipLaunchKernelGGL((attn_dq_kernel<DP, false, true>), grid, block, 0, st, a, b, slots);
        else hipLaunchKernelGGL((attn_dq_kernel<DP, false, false>), grid, block, 0, st, a, b, slots);
    }
}

template <int DP>
static void dkv(const AttnArgs &a, const AttnBwd &b, int slots, dim3 grid, hipStream_t st) {
    const dim3 block(256);
    if (a.causal) hipLaunchKernelGGL((attn_dkv_kernel<DP, true>), grid, block, 0, st, a, b, slots);
    else hipLaunchKernelGGL((attn_dkv_kernel<DP, false>), grid, block, 0, st, a, b, slots);
}

hipError_t launch_attention_bwd(const AttnArgs &a, const AttnBwd &b, hipStream_t st) {
    const long long items = (a.rows * (a.heads + a.kv) + 15) / 16;
    prof_begin(st, PROF_ATT_PREP);
    hipLaunchKernelGGL(attn_dot_kernel, dim3((unsigned)(items < 16384 ? items : 16384)), dim3(256), 0, st, a, b);
    hipLaunchKernelGGL(attn_scale_kernel, dim3((unsigned)(max(a.n_seq, 1) * a.kv)), dim3(256), 0, st, a, b);
    prof_end(st, PROF_ATT_PREP);
    const int slots = (int)att_slots(a.rows, a.n_seq, 128);
    const dim3 gq((unsigned)(((long long)slots * a.heads + 7) / 8 * 8)), gk((unsigned)(((long long)slots * a.kv + 7) / 8 * 8));
    prof_begin(st, PROF_ATT_DQ);
    if (a.d <= 32) dq<32>(a, b, slots, gq, st);
    else if (a.d <= 64) dq<64>(a, b, slots, gq, st);
    else if (a.d <= 96) dq<96>(a, b, slots, gq, st);
    else dq<128>(a, b, slots, gq, st);
    prof_end(st, PROF_ATT_DQ);
    prof_begin(st, PROF_ATT_DKV);
    if (a.d <= 32) dkv<32>(a, b, slots, gk, st);
    else if (a.d <= 64) dkv<64>(a, b, slots, gk, st);
    else if (a.d <= 96) dkv<96>(a, b, slots, gk, st);
    else dkv<128>(a, b, slots, gk, st);
    prof_end(st, PROF_ATT_DKV);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_attention_round(a, st);
}

}  // namespace ie
