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
// values: NL lanes a head, 16 elements each.
template <int NL>
__global__ __launch_bounds__(256) void attn_dot_kernel(AttnArgs p, AttnBwd b) {
    constexpr int PB = 256 / NL;
    const int lane = threadIdx.x % NL, parts = p.heads + p.kv;
    const long long total = p.rows * parts, step = (long long)gridDim.x * PB;
    for (long long i0 = (long long)blockIdx.x * PB; i0 < total; i0 += step) {
        const long long i = min(i0 + threadIdx.x / NL, total - 1);
        const long long row = i / parts;
        const int part = (int)(i - row * parts);
        const bool head = part < p.heads;
        v4i x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        if (16 * lane < p.dp) {
            x = *(const v4i *)((head ? b.dy + (row * p.heads + part) * p.dp : p.x + row * p.width + (long long)(part + p.kv) * p.dp) +
                               16 * lane);
            if (head) y = head16(b.o + (row * p.heads + part) * p.d, lane, p.d);
        }
        int dot = 0, sq = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            dot = __builtin_amdgcn_sdot4(x[k], y[k], dot, false);
            sq = __builtin_amdgcn_sdot4(x[k], x[k], sq, false);
        }
        dot = lane_reduce<NL>(dot, Add{});
        sq = lane_reduce<NL>(sq, Add{});
        if (lane || i != i0 + threadIdx.x / NL) continue;
        const int size = (bits_of((uint32_t)sq) + 1) >> 1;  // |.| < 2^size
        if (head) b.dots[row * p.heads + part] = int2{dot, size};
        else b.norm[row * p.kv + part - p.heads] = (int8_t)size;
    }
}

// The scales of the queries of one key head, a token a thread (workgroups of
// 256 tokens of a sequence, each of which finds the sequence's maxima itself),
// and for its keys the bounds that dK and dV are scaled by.
__global__ __launch_bounds__(256) void attn_scale_kernel(AttnArgs p, AttnBwd b) {
    __shared__ int sh[4][4];
    const Item it = att_item(p, 1);
    Span sp;
    int tile;
    if (!rank_tile<false>(p, it.rank, 256, sp, tile)) return;
    const int tid = threadIdx.x;
    int e_top = ATT_E_LO, n_top = -4096, r_top = -4096, o_top = E_MIN;
    for (int t = tid; t < sp.n; t += 256) {
        const long long row = sp.a + t;
        const int e = clip_e(p.xe[p.x_row ? row : 0]), nu = b.norm[row * p.kv + it.kvh] + e;
        e_top = max(e_top, e);
        n_top = max(n_top, nu);
        r_top = max(r_top, nu + e);
        o_top = max(o_top, (int)b.dye[b.dy_row ? row : 0]);
    }
    e_top = row_reduce_once<256>(e_top, Max{}, sh[0]);
    n_top = row_reduce_once<256>(n_top, Max{}, sh[1]);
    r_top = row_reduce_once<256>(r_top, Max{}, sh[2]);
    o_top = row_reduce_once<256>(o_top, Max{}, sh[3]);
    const int t = 256 * tile + tid;
    if (t >= sp.n) return;
    const long long row = sp.a + t;
    const int e = clip_e(p.xe[p.x_row ? row : 0]), eo = clip_e(b.oe[row]), ed = b.dye[b.dy_row ? row : 0];
    const float down = pow2f(max(ed - o_top, -60)), r = p.c * pow2f(e);
    int ka = -4096, kl = -4096;
    for (int g = 0; g < p.group; ++g) {
        const int h = it.kvh * p.group + g;
        const int2 d = b.dots[row * p.heads + h], st = p.stats[row * p.heads + h];
        const int delta = bits_of((uint32_t)abs(d.x)) + eo, rise = max(d.y + r_top, delta + e_top) + 1;
        AttnRow q;
        q.m = __int_as_float(st.x);
        q.r = r;
        q.dot = (float)d.x * pow2f(eo);
        q.a = (float)(1.0 / (double)(uint32_t)st.y) * down;  // a < 2^alpha
        q.s = pow2f(max(-rise, -126));
        q.e = rise + ed;
        q.o_top = o_top;
        q.ek = e;
        b.row[(long long)h * p.rows + row] = q;
        const int alpha = (__float_as_int(q.a) >> 23) - 126;
        ka = max(ka, alpha);
        kl = max(kl, alpha + e + max(d.y + n_top, delta) + 1);  // a |u| 2^e < 2^kl
    }
    b.key[(long long)it.kvh * p.rows + row] = AttnKey{(int16_t)ka, (int16_t)kl};
}

// dQ: a workgroup of four waves takes 64 queries of a head, 16 to a wave, one
// to four lanes, as in the forward pass; keys and values pass through LDS.
template <int DP, bool ROW, bool CAUSAL, int SPLIT>
__global__ __launch_bounds__(256, DP > 64 ? 2 : 3) void attn_dq_kernel(AttnArgs p, AttnBwd bw) {
    using T = HeadTile<DP, 256 / SPLIT>;
    constexpr int KS = T::KS, NE = DP / 16, BM = 64 / SPLIT, NB = SPLIT == 1 ? 2 : SPLIT;
    __shared__ __align__(16) int8_t sk[NB][T::BYTES], sv[NB][T::BYTES];
    __shared__ __align__(16) float sf[NB][64];
    const Item it = att_item(p, p.group);
    Span sp;
    int tile;
    if (!rank_tile<CAUSAL>(p, it.rank, BM, sp, tile)) return;
    const int h = it.kvh * p.group + it.gh, q0 = BM * tile;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, quad = lane >> 4;
    const int n = sp.n, qw = q0 + (SPLIT == 1 ? 16 * wave : 0), qi = qw + (lane & 15);
    const bool ok = qi < n, idle = qw >= n;
    const int8_t *base = p.x + (long long)sp.a * p.width;
    const int8_t *kh = base + (long long)(p.heads + it.kvh) * p.dp, *vh = kh + (long long)p.kv * p.dp;
    const int8_t *xe = p.xe + (ROW ? sp.a : 0);
    const long long row = sp.a + qi;
    v4i q[KS], g[KS];
    head_regs<KS>(base + (long long)qi * p.width + h * p.dp, ok, p.dp, lane, q);
    head_regs<KS>(bw.dy + (row * p.heads + h) * p.dp, ok, p.dp, lane, g);
    const AttnRow st = bw.row[(long long)h * p.rows + sp.a + min(qi, n - 1)];
    const float fe0 = pow2f(clip_e(xe[0]));
    const Poly scaled = poly(ROW ? st.s : fe0 * st.s);  // 2^-126 .. 2^60: exact products, no subnormal numbers
    const int keys = CAUSAL ? min(n, q0 + BM) : n, tiles = (keys + 63) / 64;
    const int last = CAUSAL ? min(n, qw + 16) : n;
    T k, v;
    k.init(p.width, p.dp);
    v.init(p.width, p.dp);
    float fe = 0.0f;
    const int me = SPLIT == 1 ? tid : lane;
    auto fetch = [&](int t) {
        k.fetch(kh, p.width, 64 * t, keys, p.dp);
        v.fetch(vh, p.width, 64 * t, keys, p.dp);
        if (ROW && me < 64) fe = pow2f(clip_e(xe[min(64 * t + me, n - 1)]));
    };
    auto weigh = [&](auto masked, int t, int buf, v4i &dh, v4i &dl) {
        const int lim = (CAUSAL ? qi : n - 1) - 64 * t - 4 * quad;  // keys seen: 16 z + i <= lim
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            dh[z] = 0;
            dl[z] = 0;
            if (masked.value && 64 * t + 16 * z >= last) continue;
            v4i s = {0, 0, 0, 0}, dp = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                s = mfma(T::frag_r(sk[buf], z, i, lane), q[i], s);
                dp = mfma(T::frag_r(sv[buf], z, i, lane), g[i], dp);
            }
            const float4 f = ROW ? *(const float4 *)&sf[buf][16 * z + 4 * quad] : float4{fe0, fe0, fe0, fe0};
            const float fs[4] = {f.x, f.y, f.z, f.w};
            int bits[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float w = weight(__builtin_fmaf((float)s[i], fs[i], -st.m), st.r, scaled);
                if (masked.value) w = 16 * z + i <= lim ? w : 0.0f;
                const float u = __builtin_fmaf((float)dp[i], fs[i], -st.dot);
                bits[i] = __float_as_int(ROW ? __builtin_fmaf(w * u, fs[i], RINT_128) : w * u + RINT_128);
            }
            int x, y;
            digits4(bits[0], bits[1], bits[2], bits[3], x, y);
            dh[z] = x;
            dl[z] = y;
        }
    };
    v4i hi[NE] = {}, lo[NE] = {};
    const int first = SPLIT == 1 ? 0 : wave;
    if (first < tiles) fetch(first);
    for (int t = first; t < tiles; t += SPLIT) {
        const int buf = SPLIT == 1 ? t & 1 : wave;
        if (SPLIT > 1) __builtin_amdgcn_wave_barrier();
        k.put(sk[buf]);
        v.put(sv[buf]);
        if (ROW && me < 64) sf[buf][me] = fe;
        if (t + SPLIT < tiles) fetch(t + SPLIT);
        if (SPLIT == 1) __syncthreads();
        else __builtin_amdgcn_wave_barrier();
        if (idle || 64 * t >= last) continue;
        v4i dh, dl;
        if (64 * t + 64 <= (CAUSAL ? qw + 1 : n)) weigh(Bool<false>{}, t, buf, dh, dl);
        else weigh(Bool<true>{}, t, buf, dh, dl);
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const v4i kt = T::frag_t(sk[buf], e, lane);
            hi[e] = mfma(kt, dh, hi[e]);
            lo[e] = mfma(kt, dl, lo[e]);
        }
    }
    if constexpr (SPLIT > 1) {
        gather_waves<4 * NE>((int *)&sk[0][0], hi, wave, lane);
        gather_waves<4 * NE>((int *)&sk[0][0], lo, wave, lane);
        static_assert(sizeof sk >= 3 * 4 * NE * 64 * sizeof(int), "a digit's sums fit the tiles");
        if (wave) return;
    }
    if (idle) return;
    const double rate = p.scale / (double)(uint32_t)p.stats[min(row, sp.a + n - 1ll) * p.heads + h].y;
    double y[4 * NE];
#pragma unroll
    for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[4 * e + i] = __builtin_fma((double)hi[e][i], 256.0, (double)lo[e][i]) * rate;
    store_odd(y, st.e, p.q, ok, p.d, lane, p.v16 + row * p.cols + h * p.d, p.p16 + row * p.parts + h);
}

// dK and dV: four lanes hold a key, a wave 16; queries, of every query head that
// shares them, pass through LDS 64 at a time.  SPLIT 1: a workgroup's four waves
// take 16 keys each and all the queries.  SPLIT 4: they take the same 16 keys
// and every fourth tile of queries each, staged by the wave itself, and add
// their sums up in LDS at the end (exact integers): where there are few keys,
// four times as many workgroups, which stage four times as much.
template <int DP, bool CAUSAL, int SPLIT>
__global__ __launch_bounds__(256, DP > 64 ? 1 : SPLIT > 1 ? 2 : 3) void attn_dkv_kernel(AttnArgs p, AttnBwd bw) {
    using T = HeadTile<DP, 256 / SPLIT>;
    constexpr int KS = T::KS, NE = DP / 16, KEYS = 64 / SPLIT, NB = SPLIT == 1 ? 2 : 1;
    __shared__ __align__(16) int8_t sq[NB * SPLIT][T::BYTES], sg[NB * SPLIT][T::BYTES];
    __shared__ __align__(16) float sr[NB * SPLIT][5][64];
    __shared__ int smark[2][4];
    const Item it = att_item(p, 1);
    Span sp;
    int tile;
    if (!rank_tile<CAUSAL>(p, it.rank, KEYS, sp, tile)) return;
    const int n = sp.n;
    if (CAUSAL) tile = (n + KEYS - 1) / KEYS - 1 - tile;  // the first keys meet the most queries
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, quad = lane >> 4;
    const int k0 = KEYS * tile, kw = k0 + (SPLIT == 1 ? 16 * wave : 0), kj = kw + (lane & 15);
    const bool ok = kj < n, idle = kw >= n;
    const int8_t *base = p.x + (long long)sp.a * p.width;
    const long long row = sp.a + kj;
    v4i k[KS], v[KS];
    head_regs<KS>(base + (long long)kj * p.width + (long long)(p.heads + it.kvh) * p.dp, ok, p.dp, lane, k);
    head_regs<KS>(base + (long long)kj * p.width + (long long)(p.heads + p.kv + it.kvh) * p.dp, ok, p.dp, lane, v);
    const float f = pow2f(clip_e(p.xe[p.x_row ? sp.a + min(kj, n - 1) : 0]));
    // the largest bounds of all queries (none: -4096 each), and of those that see a key
    const AttnKey *marks = bw.key + (long long)it.kvh * p.rows + sp.a;
    AttnKey all = ATT_NO_KEY, seen, seen_later = ATT_NO_KEY;
    for (int t = tid; t < n; t += 256) {
        const AttnKey x = marks[t];
        all = __builtin_elementwise_max(all, x);
        if (CAUSAL && t >= k0 + KEYS) seen_later = __builtin_elementwise_max(seen_later, x);
    }
    auto most = [](int x, int y) {
        return __builtin_bit_cast(int, __builtin_elementwise_max(__builtin_bit_cast(AttnKey, x), __builtin_bit_cast(AttnKey, y)));
    };
    all = __builtin_bit_cast(AttnKey, row_reduce_once<256>(__builtin_bit_cast(int, all), most, smark[0]));
    seen = all;
    if (CAUSAL) {
        // queries behind the tile, then those of the tile from the key's own on
        int later = row_reduce_once<256>(__builtin_bit_cast(int, seen_later), most, smark[1]);
        int own = lane < KEYS && k0 + lane < n ? __builtin_bit_cast(int, marks[k0 + lane]) : __builtin_bit_cast(int, ATT_NO_KEY);
#pragma unroll
        for (int o = 1; o < KEYS; o <<= 1) {
            const int x = __shfl_down(own, o, 64);
            own = lane + o < KEYS ? most(own, x) : own;
        }
        seen = __builtin_bit_cast(AttnKey, most(later, __shfl(own, kj - k0, 64)));
    }
    const int whole = all[1], kappa = seen[0], lambda = max(seen[1] - whole, -96);
    const int o_top = bw.row[(long long)it.kvh * p.group * p.rows + sp.a].o_top;
    const float sv = pow2f(min(-kappa, 126)), sk = pow2f(min(6 - lambda, 126));
    const int first = CAUSAL ? k0 / 64 : 0, tiles = (n + 63) / 64 - first, total = tiles * p.group;
    const int steps = SPLIT == 1 ? total : (total - wave + 3) / 4;
    T q, g;
    q.init(p.width, p.dp);
    g.init(p.heads * p.dp, p.dp);
    AttnRow rec;
    int fh = 0, ft = SPLIT == 1 ? 0 : wave;  // head and tile of the step that is fetched next
    auto wrap = [&](int &hh, int &tt) {
        while (tt >= tiles) {
            tt -= tiles;
            ++hh;
        }
    };
    if (SPLIT > 1) wrap(fh, ft);
    const int me = SPLIT == 1 ? tid : lane;
    auto fetch = [&]() {
        const int h = it.kvh * p.group + fh, t = 64 * (first + ft);
        q.fetch(base + h * p.dp, p.width, t, n, p.dp);
        g.fetch(bw.dy + ((long long)sp.a * p.heads + h) * p.dp, (long long)p.heads * p.dp, t, n, p.dp);
        if (me < 64) rec = bw.row[(long long)h * p.rows + sp.a + min(t + me, n - 1)];
        ft += SPLIT;
        wrap(fh, ft);
    };
    v4i acc[5][NE] = {};  // digits of dV (2) and dK (3), highest first
    const v4i bias = {(int)0xc0c0c0c0u, (int)0xc0c0c0c0u, (int)0xc0c0c0c0u, (int)0xc0c0c0c0u};  // -64
    auto weigh = [&](auto masked, const int8_t *lq, const int8_t *lg, const float *r, int i0, v4i (&dg)[5]) {
        // queries that see the key: i0 + 16 z + 4 quad + x in [kj, n) (causal), below n
        const int lo = kj - i0 - 4 * quad, hi = n - 1 - i0 - 4 * quad;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            if (masked.value) {
                dg[0][z] = dg[1][z] = dg[3][z] = dg[4][z] = 0;
                dg[2][z] = 0x40404040;
                if (i0 + 16 * z >= n || (CAUSAL && i0 + 16 * z + 15 < kw)) continue;
            }
            v4i s = {0, 0, 0, 0}, dp = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                s = mfma(T::frag_r(lq, z, i, lane), k[i], s);
                dp = mfma(T::frag_r(lg, z, i, lane), v[i], dp);
            }
            float r5[5][4];
#pragma unroll
            for (int y = 0; y < 5; ++y) {
                const float4 x = *(const float4 *)(r + y * 64 + 16 * z + 4 * quad);
                r5[y][0] = x.x;
                r5[y][1] = x.y;
                r5[y][2] = x.z;
                r5[y][3] = x.w;
            }
            int ab[4], cb[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float w = weight(__builtin_fmaf((float)s[x], f, -r5[0][x]), r5[1][x]);
                if (masked.value) w = 16 * z + x <= hi && (!CAUSAL || 16 * z + x >= lo) ? w : 0.0f;
                const float u = __builtin_fmaf((float)dp[x], f, -r5[2][x]);
                ab[x] = __float_as_int(__builtin_fmaf(w * r5[3][x], sv, RINT_128));
                cb[x] = __float_as_int(__builtin_fmaf(w * u * r5[4][x], sk, RINT_MAGIC + 32896.0f));
            }
            int x, y, w;
            digits4(ab[0], ab[1], ab[2], ab[3], x, y);
            dg[0][z] = x;
            dg[1][z] = y;
            digits3x4(cb[0], cb[1], cb[2], cb[3], x, y, w);
            dg[2][z] = x;
            dg[3][z] = y;
            dg[4][z] = w;
        }
    };
    if (steps > 0) fetch();
    int ct = SPLIT == 1 ? 0 : wave, ch = 0;
    if (SPLIT > 1) wrap(ch, ct);
    for (int i = 0; i < steps; ++i) {
        const int buf = SPLIT == 1 ? i & 1 : wave;
        if (SPLIT > 1) __builtin_amdgcn_wave_barrier();
        q.put(sq[buf]);
        g.put(sg[buf]);
        if (me < 64) {
            sr[buf][0][me] = rec.m;
            sr[buf][1][me] = rec.r;
            sr[buf][2][me] = rec.dot;
            sr[buf][3][me] = rec.a;
            sr[buf][4][me] = (float)((double)rec.a * pow2(rec.ek - whole));
        }
        const int i0 = 64 * (first + ct);
        ct += SPLIT;
        wrap(ch, ct);
        if (i + 1 < steps) fetch();
        if (SPLIT == 1) __syncthreads();
        else __builtin_amdgcn_wave_barrier();
        if (idle || (CAUSAL && i0 + 63 < kw)) continue;
        v4i dg[5];
        if (i0 + 64 <= n && (!CAUSAL || kw + 15 <= i0)) weigh(Bool<false>{}, sq[buf], sg[buf], &sr[buf][0][0], i0, dg);
        else weigh(Bool<true>{}, sq[buf], sg[buf], &sr[buf][0][0], i0, dg);
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const v4i gt = T::frag_t(sg[buf], e, lane), qt = T::frag_t(sq[buf], e, lane);
            acc[0][e] = mfma(gt, dg[0], acc[0][e]);
            acc[1][e] = mfma(gt, dg[1], acc[1][e]);
            acc[2][e] = mfma(qt, bias, acc[2][e]);
            acc[2][e] = mfma(qt, dg[2], acc[2][e]);
            acc[3][e] = mfma(qt, dg[3], acc[3][e]);
            acc[4][e] = mfma(qt, dg[4], acc[4][e]);
        }
    }
    if constexpr (SPLIT > 1) {
        static_assert(sizeof sq >= 3 * 4 * NE * 64 * sizeof(int), "a digit's sums fit the tiles");
#pragma unroll
        for (int a = 0; a < 5; ++a) gather_waves<4 * NE>((int *)&sq[0][0], acc[a], wave, lane);
        if (wave) return;
    }
    if (idle) return;
    double y[4 * NE];
    int16_t *out = p.v16 + row * p.cols, *need = p.p16 + row * p.parts;
#pragma unroll
    for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[4 * e + i] = ((double)acc[2][e][i] * 65536.0 + ((double)acc[3][e][i] * 256.0 + (double)acc[4][e][i])) * p.scale;
    store_odd(y, lambda - 6 + whole + o_top, p.q, ok, p.d, lane, out + (p.heads + it.kvh) * p.d, need + p.heads + it.kvh);
#pragma unroll
    for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[4 * e + i] = (double)acc[0][e][i] * 256.0 + (double)acc[1][e][i];
    store_odd(y, kappa + o_top, p.q, ok, p.d, lane, out + (p.heads + p.kv + it.kvh) * p.d, need + p.heads + p.kv + it.kvh);
}

template <int DP, int SPLIT>
static void dq(AttnArgs a, const AttnBwd &b, hipStream_t st) {
    a.chunk = att_chunk(a, 64 / SPLIT, !a.causal);
    const dim3 grid(att_grid(att_slots(a.rows, a.n_seq, 64 / SPLIT), a.kv, a.group)), block(256);
    if (a.x_row) {
        if (a.causal) hipLaunchKernelGGL((attn_dq_kernel<DP, true, true, SPLIT>), grid, block, 0, st, a, b);
        else hipLaunchKernelGGL((attn_dq_kernel<DP, true, false, SPLIT>), grid, block, 0, st, a, b);
    } else {
        if (a.causal) hipLaunchKernelGGL((attn_dq_kernel<DP, false, true, SPLIT>), grid, block, 0, st, a, b);
        else hipLaunchKernelGGL((attn_dq_kernel<DP, false, false, SPLIT>), grid, block, 0, st, a, b);
    }
}

template <int DP>
static void dq(const AttnArgs &a, const AttnBwd &b, hipStream_t st) {
    if (att_slots(a.rows, a.n_seq, 64) * a.heads < 2 * NCU) dq<DP, 4>(a, b, st);
    else dq<DP, 1>(a, b, st);
}

template <int DP>
static void dkv(AttnArgs a, const AttnBwd &b, int split, hipStream_t st) {
    a.chunk = att_chunk(a, 64 / split, !a.causal);
    const dim3 grid(att_grid(att_slots(a.rows, a.n_seq, 64 / split), a.kv, 1)), block(256);
    if (split == 1) {
        if (a.causal) hipLaunchKernelGGL((attn_dkv_kernel<DP, true, 1>), grid, block, 0, st, a, b);
        else hipLaunchKernelGGL((attn_dkv_kernel<DP, false, 1>), grid, block, 0, st, a, b);
    } else {
        if (a.causal) hipLaunchKernelGGL((attn_dkv_kernel<DP, true, 4>), grid, block, 0, st, a, b);
        else hipLaunchKernelGGL((attn_dkv_kernel<DP, false, 4>), grid, block, 0, st, a, b);
    }
}

hipError_t launch_attention_bwd(const AttnArgs &a, const AttnBwd &b, hipStream_t st) {
    const int nl = a.dp <= 16 ? 1 : a.dp <= 32 ? 2 : a.dp <= 64 ? 4 : 8;
    const long long items = (a.rows * (a.heads + a.kv) + 256 / nl - 1) / (256 / nl);
    const dim3 gd((unsigned)(items < 8 * NCU ? items : 8 * NCU)), block(256);
    prof_begin(st, PROF_ATT_PREP);
    if (nl == 1) hipLaunchKernelGGL(attn_dot_kernel<1>, gd, block, 0, st, a, b);
    else if (nl == 2) hipLaunchKernelGGL(attn_dot_kernel<2>, gd, block, 0, st, a, b);
    else if (nl == 4) hipLaunchKernelGGL(attn_dot_kernel<4>, gd, block, 0, st, a, b);
    else hipLaunchKernelGGL(attn_dot_kernel<8>, gd, block, 0, st, a, b);
    AttnArgs c = a;
    c.chunk = att_chunk(a, 256, true);
    hipLaunchKernelGGL(attn_scale_kernel, dim3(att_grid(att_slots(a.rows, a.n_seq, 256), a.kv, 1)), block, 0, st, c, b);
    prof_end(st, PROF_ATT_PREP);
    prof_begin(st, PROF_ATT_DQ);
    if (a.d <= 32) dq<32>(a, b, st);
    else if (a.d <= 64) dq<64>(a, b, st);
    else if (a.d <= 96) dq<96>(a, b, st);
    else dq<128>(a, b, st);
    prof_end(st, PROF_ATT_DQ);
    const int split = att_slots(a.rows, a.n_seq, 64) * a.kv < 4 * NCU ? 4 : 1;
    prof_begin(st, PROF_ATT_DKV);
    if (a.d <= 32) dkv<32>(a, b, split, st);
    else if (a.d <= 64) dkv<64>(a, b, split, st);
    else if (a.d <= 96) dkv<96>(a, b, split, st);
    else dkv<128>(a, b, split, st);
    prof_end(st, PROF_ATT_DKV);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_attention_round(a, st);
}

}  // namespace ie
