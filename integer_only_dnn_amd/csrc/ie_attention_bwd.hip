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
// a root mean square of four units.  All of it runs on exponents relative to the
// sequence's largest one, so that a sequence of the smallest exponents is as exact as any
// (a score's two factors take that power of two between them).  Rows of fine weights (ie_attn.h) have theirs with
// 2^14 in the place of 1 and 2^6, and so have the keys that share a sequence and
// a key head with one: four digits, |n| <= 2^14 32512.
#include "ie_attn.h"

#pragma clang fp contract(off)

namespace ie {

__device__ __forceinline__ int bits_of(uint32_t n) { return 32 - __clz((int)n); }  // n = 0: 0

// A row's products of dO with O and itself by head, and the norms of its
// values: NL lanes a head, 16 elements each.  A stream over dO, O and V: 58 MB of
// 25216 tokens x 12 heads of 64 in 11.5 us.
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

// O's exponents, relative: below those of V where its mantissas cancel, above them where they have fewer bits.
constexpr int O_E_LO = -126, O_E_HI = 40;
// 2^(e - top), a key's factor.
__device__ __forceinline__ float rel_pow2(int e, int top) { return pow2_down(clip_e(e) - top); }

// The scales of the queries of one key head, a token a thread (workgroups of
// 256 tokens of a sequence, each of which finds the sequence's maxima itself),
// and for its keys the bounds that dK and dV are scaled by.  Bound by the round
// trips to memory of a workgroup: 9.9 us at 128 x 197 tokens x 12 heads, 7.5 at
// 4096 x 4.
__global__ __launch_bounds__(256) void attn_scale_kernel(AttnArgs p, AttnBwd b) {
    __shared__ int sh[4][4];
    const Item it = att_item(p, 1);
    Span sp;
    int tile;
    if (!rank_tile<false>(p, it.rank, 256, sp, tile)) return;
    const int tid = threadIdx.x;
    int e_top = ATT_E_LO, n_top = -4096, r_top = -4096, o_top = E_MIN;
#pragma unroll 4
    for (int t = tid; t < sp.n; t += 256) {
        const long long row = sp.a + t;
        const int e = clip_e(p.xe[p.x_row ? row : 0]), nu = b.norm[row * p.kv + it.kvh] + e;
        e_top = max(e_top, e);
        n_top = max(n_top, nu);
        r_top = max(r_top, nu + e);
        o_top = max(o_top, (int)b.dye[b.dy_row ? row : 0]);
    }
    e_top = row_reduce_once<256>(e_top, Max{}, sh[0]);
    n_top = row_reduce_once<256>(n_top, Max{}, sh[1]) - e_top;
    r_top = row_reduce_once<256>(r_top, Max{}, sh[2]) - 2 * e_top;
    o_top = row_reduce_once<256>(o_top, Max{}, sh[3]);
    const int t = 256 * tile + tid;
    if (t >= sp.n) return;
    const long long row = sp.a + t;
    const int e = clip_e(p.xe[p.x_row ? row : 0]), eo = min(max((int)b.oe[row] - e_top, O_E_LO), O_E_HI);
    const int ed = b.dye[b.dy_row ? row : 0];
    const float down = pow2f(max(ed - o_top, -60)), r = p.c * pow2f(e) * pow2f(e_top);
    int ka = -4096, kl = -4096, fine = 0;
    for (int g = 0; g < p.group; ++g) {
        const int h = it.kvh * p.group + g;
        const int2 d = b.dots[row * p.heads + h], st = p.stats[row * p.heads + h];
        const int delta = bits_of((uint32_t)abs(d.x)) + eo, rise = max(d.y + r_top, delta) + 1;
        AttnRow q;
        q.m = __int_as_float(st.x & ~1) * pow2f(-e_top);  // the last bit: a row of fine weights
        fine |= st.x & 1;
        q.r = r;
        q.dot = (float)d.x * pow2f(eo);
        q.a = (float)(1.0 / (double)(uint32_t)st.y) * down;  // a < 2^alpha
        q.s = pow2f(-rise);
        q.e = rise + ed + 2 * e_top;
        q.tops = o_top << 8 | (e_top & 0xff);
        q.ek = e - e_top;
        b.row[(long long)h * p.rows + row] = q;
        const int alpha = (__float_as_int(q.a) >> 23) - 126;
        ka = max(ka, alpha);
        kl = max(kl, alpha + e - e_top + max(d.y + n_top, delta) + 1);  // a |u| 2^e < 2^kl
    }
    b.key[(long long)it.kvh * p.rows + row] = AttnKey{(int16_t)ka, (int16_t)kl};
    if (fine) p.flags[FINE_WORD] = 1;  // the same from every thread that says so
}

// The largest bounds of all queries of a sequence (none: -4096 each), and of those that see
// key kj of the tile of KEYS from k0 on.
template <bool CAUSAL, int KEYS>
__device__ __forceinline__ void key_bounds(const AttnKey *marks, int n, int k0, int kj, int (&sh)[2][4], AttnKey &all, AttnKey &seen) {
    const int tid = threadIdx.x, lane = tid & 63;
    AttnKey seen_later = ATT_NO_KEY;
    all = ATT_NO_KEY;
#pragma unroll 4
    for (int t = tid; t < n; t += 256) {
        const AttnKey x = marks[t];
        all = __builtin_elementwise_max(all, x);
        if (CAUSAL && t >= k0 + KEYS) seen_later = __builtin_elementwise_max(seen_later, x);
    }
    auto most = [](int x, int y) {
        return __builtin_bit_cast(int, __builtin_elementwise_max(__builtin_bit_cast(AttnKey, x), __builtin_bit_cast(AttnKey, y)));
    };
    all = __builtin_bit_cast(AttnKey, row_reduce_once<256>(__builtin_bit_cast(int, all), most, sh[0]));
    seen = all;
    if (CAUSAL) {
        // queries behind the tile, then those of the tile from the key's own on
        int later = row_reduce_once<256>(__builtin_bit_cast(int, seen_later), most, sh[1]);
        int own = lane < KEYS && k0 + lane < n ? __builtin_bit_cast(int, marks[k0 + lane]) : __builtin_bit_cast(int, ATT_NO_KEY);
#pragma unroll
        for (int o = 1; o < KEYS; o <<= 1) {
            const int x = __shfl_down(own, o, 64);
            own = lane + o < KEYS ? most(own, x) : own;
        }
        seen = __builtin_bit_cast(AttnKey, most(later, __shfl(own, kj - k0, 64)));
    }
}

// dQ: a workgroup of four waves takes 64 queries of a head, 16 to a wave, one
// to four lanes, as in the forward pass; keys and values pass through LDS.  SPLIT
// 4: the waves take the same 16 queries and every fourth tile of keys each, and
// add their sums up at the end.
// Bound by vector instructions (17 to a weight, 29 and 20 to a pair of tokens with all that
// lies around them), 75 % of the cycles in which a CU is busy at 128 x 197 tokens x 12
// heads of 64 (72 us), and by the longest rows' way through their keys where tiles are
// few (4096 tokens in 3 sequences x 16 heads, causal: 51 us, 74 %).
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
    const int e_top = (int8_t)st.tops;
    const float fe0 = 1.0f;  // where all rows share an exponent
    const Poly scaled = poly(st.s);  // 2^-70 .. 2^-1: exact products, no subnormal numbers
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
        if (ROW && me < 64) fe = rel_pow2(xe[min(64 * t + me, n - 1)], e_top);
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
// shares them, pass through LDS 64 at a time.  By SPLIT:
// 1: a workgroup's four waves take 16 keys each and all the queries and elements.
// 4: they take the same 16 keys and every fourth tile of queries each, staged by
//    the wave itself, and add their sums up in LDS at the end (exact integers):
//    where there are few keys, four times as many workgroups, which stage four
//    times as much.
// 2: two take 16 keys and half of a tile's queries each, the digits of 32 keys and
//    64 queries change hands in LDS, and each wave sums a quarter of the elements:
//    half the registers for the sums (five digits to an element and key), which are
//    160 to a lane otherwise where heads have 128 elements.
// Bound by vector instructions (21 to a weight, 48 to a pair at 197 tokens and 32 at up
// to 2230, with masked pairs, the marks and the results in fp64, beside a sixth of the time
// in matrix instructions) and, at two to three waves a SIMD, by waits for LDS:
// 128 x 197 tokens x 12 heads of 64 70 % of the cycles in which a CU is busy, 125 us.
template <int DP, bool CAUSAL, int SPLIT>
__global__ __launch_bounds__(256, SPLIT == 2 ? 2 : DP > 64 ? 1 : SPLIT == 4 ? 2 : 3) void attn_dkv_kernel(AttnArgs p, AttnBwd bw) {
    constexpr bool OWN = SPLIT == 4, SHARE = SPLIT == 2;  // own tiles; shared elements
    using T = HeadTile<DP, OWN ? 64 : 256>;
    constexpr int KS = T::KS, NE = DP / 16, KEYS = 64 / SPLIT, NB = OWN ? 4 : 2;
    constexpr int KG = SHARE ? 2 : 1, ME = SHARE ? (NE + 3) / 4 : NE, NZ = SHARE ? 2 : 4;  // of a wave
    __shared__ __align__(16) int8_t sq[NB][T::BYTES], sg[NB][T::BYTES];
    __shared__ __align__(16) float sr[NB][5][64];
    __shared__ __align__(16) int sd[SHARE ? 5 : 1][KG][16][4][4];  // digits: keys, lane group, queries
    __shared__ int smark[2][4];
    const Item it = att_item(p, 1);
    Span sp;
    int tile;
    if (!rank_tile<CAUSAL>(p, it.rank, KEYS, sp, tile)) return;
    const int n = sp.n;
    if (CAUSAL) tile = (n + KEYS - 1) / KEYS - 1 - tile;  // the first keys meet the most queries
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, quad = lane >> 4;
    const int k0 = KEYS * tile, kw = k0 + (OWN ? 0 : 16 * (wave % (KEYS / 16))), kj = kw + (lane & 15);
    const bool ok = kj < n, idle = kw >= n;
    const int8_t *base = p.x + (long long)sp.a * p.width;
    const long long row = sp.a + kj;
    v4i k[KS], v[KS];
    head_regs<KS>(base + (long long)kj * p.width + (long long)(p.heads + it.kvh) * p.dp, ok, p.dp, lane, k);
    head_regs<KS>(base + (long long)kj * p.width + (long long)(p.heads + p.kv + it.kvh) * p.dp, ok, p.dp, lane, v);
    AttnKey all, seen;
    key_bounds<CAUSAL, KEYS>(bw.key + (long long)it.kvh * p.rows + sp.a, n, k0, kj, smark, all, seen);
    const int whole = all[1], kappa = seen[0], lambda = max(seen[1] - whole, -96);
    const int tops = bw.row[(long long)it.kvh * p.group * p.rows + sp.a].tops, o_top = tops >> 8, e_top = (int8_t)tops;
    const float f = rel_pow2(p.xe[p.x_row ? sp.a + min(kj, n - 1) : 0], e_top);
    const float sv = pow2f(min(-kappa, 126)), sk = pow2f(min(6 - lambda, 126));
    const int first = CAUSAL ? k0 / 64 : 0, tiles = (n + 63) / 64 - first, total = tiles * p.group;
    const int steps = OWN ? (total - wave + 3) / 4 : total, z0 = SHARE ? 2 * (wave >> 1) : 0;
    T q, g;
    q.init(p.width, p.dp);
    g.init(p.heads * p.dp, p.dp);
    AttnRow rec;
    int fh = 0, ft = OWN ? wave : 0;  // head and tile of the step that is fetched next
    auto wrap = [&](int &hh, int &tt) {
        while (tt >= tiles) {
            tt -= tiles;
            ++hh;
        }
    };
    if (OWN) wrap(fh, ft);
    const int me = OWN ? lane : tid;
    auto fetch = [&]() {
        const int h = it.kvh * p.group + fh, t = 64 * (first + ft);
        q.fetch(base + h * p.dp, p.width, t, n, p.dp);
        g.fetch(bw.dy + ((long long)sp.a * p.heads + h) * p.dp, (long long)p.heads * p.dp, t, n, p.dp);
        if (me < 64) rec = bw.row[(long long)h * p.rows + sp.a + min(t + me, n - 1)];
        ft += OWN ? 4 : 1;
        wrap(fh, ft);
    };
    v4i acc[KG][5][ME] = {};  // digits of dV (2) and dK (3), highest first
    auto weigh = [&](auto masked, const int8_t *lq, const int8_t *lg, const float *r, int i0, v4i (&dg)[5]) {
        // queries that see the key: i0 + 16 z + 4 quad + x in [kj, n) (causal), below n
        const int lo = kj - i0 - 4 * quad, hi = n - 1 - i0 - 4 * quad;
#pragma unroll
        for (int zi = 0; zi < NZ; ++zi) {
            const int z = z0 + zi;
            if (masked.value) {
#pragma unroll
                for (int y = 0; y < 5; ++y) dg[y][zi] = 0;
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
            dg[0][zi] = x;
            dg[1][zi] = y;
            digits3x4(cb[0], cb[1], cb[2], cb[3], x, y, w);
            dg[2][zi] = x;
            dg[3][zi] = y;
            dg[4][zi] = w;
        }
    };
    if (steps > 0) fetch();
    int ct = OWN ? wave : 0, ch = 0;
    if (OWN) wrap(ch, ct);
    for (int i = 0; i < steps; ++i) {
        const int buf = OWN ? wave : i & 1;
        if (OWN) __builtin_amdgcn_wave_barrier();
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
        ct += OWN ? 4 : 1;
        wrap(ch, ct);
        if (i + 1 < steps) fetch();
        if (OWN) __builtin_amdgcn_wave_barrier();
        else __syncthreads();
        const bool none = idle || (CAUSAL && i0 + 63 < kw);
        if (!SHARE && none) continue;
        v4i dg[5];
        if (SHARE && none) {
#pragma unroll
            for (int y = 0; y < 5; ++y) dg[y] = v4i{0, 0, 0, 0};
        } else if (i0 + 64 <= n && (!CAUSAL || kw + 15 <= i0)) {
            weigh(Bool<false>{}, sq[buf], sg[buf], &sr[buf][0][0], i0, dg);
        } else {
            weigh(Bool<true>{}, sq[buf], sg[buf], &sr[buf][0][0], i0, dg);
        }
        if constexpr (SHARE) {
            // the digits of 32 keys change hands: a wave sums a quarter of the elements
#pragma unroll
            for (int y = 0; y < 5; ++y) *(int2 *)&sd[y][wave & 1][lane & 15][quad][z0] = int2{dg[y][0], dg[y][1]};
            __syncthreads();
        }
#pragma unroll
        for (int g2 = 0; g2 < KG; ++g2) {
            if constexpr (SHARE) {
#pragma unroll
                for (int y = 0; y < 5; ++y) dg[y] = *(const v4i *)sd[y][g2][lane & 15][quad];
            }
#pragma unroll
            for (int e = 0; e < ME; ++e) {
                const int at = SHARE ? wave + 4 * e : e;
                if (SHARE && NE % 4 && at >= NE) continue;
                const v4i gt = T::frag_t(sg[buf], at, lane), qt = T::frag_t(sq[buf], at, lane);
                acc[g2][0][e] = mfma(gt, dg[0], acc[g2][0][e]);
                acc[g2][1][e] = mfma(gt, dg[1], acc[g2][1][e]);
#pragma unroll
                for (int y = 2; y < 5; ++y) acc[g2][y][e] = mfma(qt, dg[y], acc[g2][y][e]);
            }
        }
    }
    if constexpr (OWN) {
        static_assert(sizeof sq >= 3 * 4 * NE * 64 * sizeof(int), "a digit's sums fit the tiles");
#pragma unroll
        for (int a = 0; a < 5; ++a) gather_waves<4 * NE>((int *)&sq[0][0], acc[0][a], wave, lane);
        if (wave) return;
    }
    if (!SHARE && idle) return;
    const int head_k = p.heads + it.kvh, head_v = head_k + p.kv, e_k = lambda - 6 + whole + 2 * e_top + o_top, e_v = kappa + o_top;
    auto value = [&](int g2, bool of_k, int e, int i) {
        const auto &a = acc[g2];
        return of_k ? ((double)a[2][e][i] * 65536.0 + ((double)a[3][e][i] * 256.0 + (double)a[4][e][i])) * p.scale
                    : (double)a[0][e][i] * 256.0 + (double)a[1][e][i];
    };
    if constexpr (!SHARE) {
        double y[4 * NE];
        int16_t *out = p.v16 + row * p.cols, *need = p.p16 + row * p.parts;
#pragma unroll
        for (int of_v = 0; of_v < 2; ++of_v) {
#pragma unroll
            for (int i = 0; i < 4 * NE; ++i) y[i] = value(0, !of_v, i >> 2, i & 3);
            const int head = of_v ? head_v : head_k;
            store_odd(y, of_v ? e_v : e_k, p.q, ok, p.d, lane, out + head * p.d, need + head);
        }
    } else {
        // a head's need is that of four waves' elements; kappa and lambda are those of a key, in lanes of its group
        __shared__ int sm[4][2][2][16], se[2][2][16];
        if (lane < 16) {
            se[0][wave & 1][lane] = e_k;
            se[1][wave & 1][lane] = e_v;
        }
        auto values = [&](int g2, int of_v, double (&y)[4 * ME]) {
#pragma unroll
            for (int i = 0; i < 4 * ME; ++i) y[i] = value(g2, !of_v, i >> 2, i & 3);  // zeros past the head
        };
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            double y[4 * ME];
            values(x >> 1, x & 1, y);
            const int w = max_word(y);
            if (lane < 16) sm[wave][x >> 1][x & 1][lane] = w;
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int g2 = x >> 1, of_v = x & 1, c = lane & 15, key = k0 + 16 * g2 + c, head = of_v ? head_v : head_k;
            double y[4 * ME];
            values(g2, of_v, y);
            const int w = max(max(sm[0][g2][of_v][c], sm[1][g2][of_v][c]), max(sm[2][g2][of_v][c], sm[3][g2][of_v][c]));
            const int need = need_word(w, p.q);
            const double inv = odd_scale(need);
            if (key < n && tid < 16)
                p.p16[(sp.a + key) * (long long)p.parts + head] = (int16_t)(need == NEED_NONE ? P_NONE : need + se[of_v][g2][c]);
#pragma unroll
            for (int e = 0; e < ME; ++e) {
                const int at = 16 * (wave + 4 * e) + 4 * quad;
                if (at < DP) write_odd(y + 4 * e, inv, key < n, at, p.d, p.v16 + (sp.a + key) * (long long)p.cols + head * p.d);
            }
        }
    }
}

// The same with fine weights: dQ of the rows that the forward pass has marked, and dK
// and dV of their sequences and key heads, in four digits (dV first, then dK: their
// sums in the same registers), into the places that the kernels above have
// filled.  A call without such a row ends at its first load.
template <int DP>
struct FineLds {
    using T = HeadTile<DP>;
    int8_t a[2][T::BYTES], b[2][T::BYTES];
    float f[2][5][64];
    int mark[2][4], any[4];
};

// Whether a thread of the workgroup says so; the workgroup's LDS is free behind it.
__device__ __forceinline__ bool any_of(bool mine, int (&sh)[4]) {
    const bool some = __ballot(mine) != 0;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = some;
    __syncthreads();
    return sh[0] | sh[1] | sh[2] | sh[3];
}

template <int DP, bool CAUSAL>
__device__ __forceinline__ void fine_dq(const AttnArgs &p, const AttnBwd &bw, int idx, int of_q, FineLds<DP> &lds) {
    using T = HeadTile<DP>;
    constexpr int KS = T::KS, NE = DP / 16;
    const Item it = att_item(p, p.group, idx, of_q);
    const int kvh = it.kvh, h = kvh * p.group + it.gh;
    Span sp;
    int tile;
    if (!rank_tile<CAUSAL>(p, it.rank, 64, sp, tile)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, quad = lane >> 4;
    const int n = sp.n, q0 = 64 * tile, qi = q0 + 16 * wave + (lane & 15);
    const long long row = sp.a + qi;
    const bool fine = qi < n && (p.stats[row * p.heads + h].x & 1);
    if (!any_of(fine, lds.any)) return;
    const int8_t *base = p.x + (long long)sp.a * p.width;
    const int8_t *kh = base + (long long)(p.heads + kvh) * p.dp, *vh = kh + (long long)p.kv * p.dp;
    v4i q[KS], g[KS];
    head_regs<KS>(base + (long long)qi * p.width + h * p.dp, qi < n, p.dp, lane, q);
    head_regs<KS>(bw.dy + (row * p.heads + h) * p.dp, qi < n, p.dp, lane, g);
    const AttnRow st = bw.row[(long long)h * p.rows + sp.a + min(qi, n - 1)];
    const int e_top = (int8_t)st.tops;
    const Poly scaled = poly(st.s);
    const int keys = CAUSAL ? min(n, q0 + 64) : n, tiles = (keys + 63) / 64, lim = CAUSAL ? qi : n - 1;
    T k, v;
    k.init(p.width, p.dp);
    v.init(p.width, p.dp);
    float fe = 0.0f;
    auto fetch = [&](int t) {
        k.fetch(kh, p.width, 64 * t, keys, p.dp);
        v.fetch(vh, p.width, 64 * t, keys, p.dp);
        if (tid < 64) fe = rel_pow2(p.xe[p.x_row ? sp.a + min(64 * t + tid, n - 1) : 0], e_top);
    };
    v4i acc[4][NE] = {};
    fetch(0);
    for (int t = 0; t < tiles; ++t) {
        const int buf = t & 1;
        k.put(lds.a[buf]);
        v.put(lds.b[buf]);
        if (tid < 64) lds.f[buf][0][tid] = fe;
        if (t + 1 < tiles) fetch(t + 1);
        __syncthreads();
        v4i dg[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            v4i s = {0, 0, 0, 0}, dp = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                s = mfma(T::frag_r(lds.a[buf], z, i, lane), q[i], s);
                dp = mfma(T::frag_r(lds.b[buf], z, i, lane), g[i], dp);
            }
            int n4[4], o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = lds.f[buf][0][16 * z + 4 * quad + i];
                float w = weight(__builtin_fmaf((float)s[i], f, -st.m), st.r, scaled);
                w = 64 * t + 16 * z + 4 * quad + i <= lim ? w : 0.0f;
                const float u = __builtin_fmaf((float)dp[i], f, -st.dot);
                n4[i] = (int)__builtin_rintf(w * u * f * FINE_UNIT);
            }
            digits4x4(n4, o);
#pragma unroll
            for (int y = 0; y < 4; ++y) dg[y][z] = o[y];
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const v4i kt = T::frag_t(lds.a[buf], e, lane);
#pragma unroll
            for (int y = 0; y < 4; ++y) acc[y][e] = mfma(kt, dg[y], acc[y][e]);
        }
    }
    const double rate = p.scale / (double)(uint32_t)p.stats[(sp.a + min(qi, n - 1)) * (long long)p.heads + h].y;
    double y[4 * NE];
#pragma unroll
    for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[4 * e + i] = whole4(acc[0][e][i], acc[1][e][i], acc[2][e][i], acc[3][e][i]) * rate;
    store_odd(y, st.e - ATT_FINE, p.q, fine, p.d, lane, p.v16 + row * p.cols + h * p.d, p.p16 + row * p.parts + h);
}

template <int DP, bool CAUSAL>
__device__ __forceinline__ void fine_dkv(const AttnArgs &p, const AttnBwd &bw, int idx, FineLds<DP> &lds) {
    using T = HeadTile<DP>;
    constexpr int KS = T::KS, NE = DP / 16;
    const int kvh = idx % p.kv;
    Span sp;
    int tile;
    if (!rank_tile<CAUSAL>(p, idx / p.kv, 64, sp, tile)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, quad = lane >> 4;
    const int n = sp.n;
    bool fine = false;
    for (int t = tid; t < n; t += 256)
        for (int g = 0; g < p.group; ++g) fine |= p.stats[(long long)(sp.a + t) * p.heads + kvh * p.group + g].x & 1;
    if (!any_of(fine, lds.any)) return;
    if (CAUSAL) tile = (n + 63) / 64 - 1 - tile;
    const int k0 = 64 * tile, kj = k0 + 16 * wave + (lane & 15);
    const bool ok = kj < n;
    const int8_t *base = p.x + (long long)sp.a * p.width;
    const long long row = sp.a + kj;
    v4i k[KS], v[KS];
    head_regs<KS>(base + (long long)kj * p.width + (long long)(p.heads + kvh) * p.dp, ok, p.dp, lane, k);
    head_regs<KS>(base + (long long)kj * p.width + (long long)(p.heads + p.kv + kvh) * p.dp, ok, p.dp, lane, v);
    AttnKey all, seen;
    key_bounds<CAUSAL, 64>(bw.key + (long long)kvh * p.rows + sp.a, n, k0, kj, lds.mark, all, seen);
    const int whole = all[1], kappa = seen[0], lambda = max(seen[1] - whole, -96);
    const int tops = bw.row[(long long)kvh * p.group * p.rows + sp.a].tops, o_top = tops >> 8, e_top = (int8_t)tops;
    const float f = rel_pow2(p.xe[p.x_row ? sp.a + min(kj, n - 1) : 0], e_top);
    const int first = CAUSAL ? k0 / 64 : 0, tiles = (n + 63) / 64 - first, steps = tiles * p.group;
    T q, g;
    q.init(p.width, p.dp);
    g.init(p.heads * p.dp, p.dp);
    auto sweep = [&](auto of_k) {
        const float unit = pow2f(min(ATT_FINE - (of_k.value ? lambda : kappa), 126));
        AttnRow rec;
        auto fetch = [&](int i) {
            const int h = kvh * p.group + i / tiles, t = 64 * (first + i % tiles);
            q.fetch(base + h * p.dp, p.width, t, n, p.dp);
            g.fetch(bw.dy + ((long long)sp.a * p.heads + h) * p.dp, (long long)p.heads * p.dp, t, n, p.dp);
            if (tid < 64) rec = bw.row[(long long)h * p.rows + sp.a + min(t + tid, n - 1)];
        };
        v4i acc[4][NE] = {};
        fetch(0);
        for (int i = 0; i < steps; ++i) {
            const int buf = i & 1, i0 = 64 * (first + i % tiles);
            q.put(lds.a[buf]);
            g.put(lds.b[buf]);
            if (tid < 64) {
                lds.f[buf][0][tid] = rec.m;
                lds.f[buf][1][tid] = rec.r;
                lds.f[buf][2][tid] = rec.dot;
                lds.f[buf][3][tid] = rec.a;
                lds.f[buf][4][tid] = (float)((double)rec.a * pow2(rec.ek - whole));
            }
            if (i + 1 < steps) fetch(i + 1);
            __syncthreads();
            v4i dg[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                v4i s = {0, 0, 0, 0}, dp = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                    s = mfma(T::frag_r(lds.a[buf], z, c, lane), k[c], s);
                    if (of_k.value) dp = mfma(T::frag_r(lds.b[buf], z, c, lane), v[c], dp);
                }
                int n4[4], o[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = 16 * z + 4 * quad + x, query = i0 + j;
                    float w = weight(__builtin_fmaf((float)s[x], f, -lds.f[buf][0][j]), lds.f[buf][1][j]);
                    w = query < n && (!CAUSAL || query >= kj) ? w : 0.0f;
                    const float u = __builtin_fmaf((float)dp[x], f, -lds.f[buf][2][j]);
                    n4[x] = (int)__builtin_rintf((of_k.value ? w * u * lds.f[buf][4][j] : w * lds.f[buf][3][j]) * unit);
                }
                digits4x4(n4, o);
#pragma unroll
                for (int y = 0; y < 4; ++y) dg[y][z] = o[y];
            }
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                const v4i xt = T::frag_t(of_k.value ? lds.a[buf] : lds.b[buf], e, lane);
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[y][e] = mfma(xt, dg[y], acc[y][e]);
            }
        }
        double y[4 * NE];
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[4 * e + i] = whole4(acc[0][e][i], acc[1][e][i], acc[2][e][i], acc[3][e][i]);
                if (of_k.value) y[4 * e + i] *= p.scale;
            }
        const int head = p.heads + kvh + (of_k.value ? 0 : p.kv), e = (of_k.value ? lambda + whole + 2 * e_top : kappa) + o_top - ATT_FINE;
        store_odd(y, e, p.q, ok, p.d, lane, p.v16 + row * p.cols + head * p.d, p.p16 + row * p.parts + head);
        __syncthreads();  // the tiles are read
    };
    sweep(Bool<false>{});
    sweep(Bool<true>{});
}

template <int DP, bool CAUSAL>
__global__ __launch_bounds__(256, DP > 64 ? 1 : 2) void attn_bwd_fine_kernel(AttnArgs p, AttnBwd bw, int of_q, int of_k) {
    __shared__ __align__(16) FineLds<DP> lds;
    if (!p.flags[FINE_WORD]) return;
    for (int idx = blockIdx.x; idx < of_q + of_k; idx += gridDim.x) {
        __syncthreads();
        if (idx < of_k) fine_dkv<DP, CAUSAL>(p, bw, idx, lds);
        else fine_dq<DP, CAUSAL>(p, bw, idx - of_k, of_q, lds);
    }
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

// Tiles split where they are fewer than two a CU (us, tokens x heads of 64, causal,
// split and whole): 1024 x 8 12 and 21; 2048 x 16 (528 tiles) 39 and 45, all keys
// seen 60 and 46; 4096 x 16 in 3 sequences 66 and 51.
template <int DP>
static void dq(const AttnArgs &a, const AttnBwd &b, hipStream_t st) {
    if (att_slots(a.rows, a.n_seq, 64) * a.heads < 2 * NCU) dq<DP, 4>(a, b, st);
    else dq<DP, 1>(a, b, st);
}

template <int DP, int SPLIT>
static void dkv(AttnArgs a, const AttnBwd &b, hipStream_t st) {
    a.chunk = att_chunk(a, 64 / SPLIT, !a.causal);
    const dim3 grid(att_grid(att_slots(a.rows, a.n_seq, 64 / SPLIT), a.kv, 1)), block(256);
    if (a.causal) hipLaunchKernelGGL((attn_dkv_kernel<DP, true, SPLIT>), grid, block, 0, st, a, b);
    else hipLaunchKernelGGL((attn_dkv_kernel<DP, false, SPLIT>), grid, block, 0, st, a, b);
}

// SPLIT 4 where there are few tiles (us, tokens x key heads, causal).  Heads of
// 64: 4096 x 4, group of 4, 82 and with SPLIT 1 277; 25216 x 12 (128 sequences,
// not causal) 315 and 129.  Heads of 128: 2048 x 2 98 and with SPLIT 2 195; 1024 x
// 8 38 and 32; 4096 x 8, group of 4, 823 and 628 (SPLIT 1, at 440 registers one
// wave a SIMD, 714).
template <int DP>
static void dkv(const AttnArgs &a, const AttnBwd &b, hipStream_t st) {
    const bool few = DP > 64 ? att_slots(a.rows, a.n_seq, 32) * a.kv < NCU : att_slots(a.rows, a.n_seq, 64) * a.kv < 4 * NCU;
    if (few) dkv<DP, 4>(a, b, st);
    else dkv<DP, (DP > 64 ? 2 : 1)>(a, b, st);
}

template <int DP>
static void bwd_fine(const AttnArgs &a, const AttnBwd &b, hipStream_t st) {
    const long long slots = att_slots(a.rows, a.n_seq, 64);
    const unsigned of_q = att_grid(slots, a.kv, a.group), of_k = (unsigned)(slots * a.kv), items = of_q + of_k;
    const dim3 grid(items < 2 * NCU ? items : 2 * NCU), block(256);
    if (a.causal) hipLaunchKernelGGL((attn_bwd_fine_kernel<DP, true>), grid, block, 0, st, a, b, (int)of_q, (int)of_k);
    else hipLaunchKernelGGL((attn_bwd_fine_kernel<DP, false>), grid, block, 0, st, a, b, (int)of_q, (int)of_k);
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
    prof_begin(st, PROF_ATT_DKV);
    if (a.d <= 32) dkv<32>(a, b, st);
    else if (a.d <= 64) dkv<64>(a, b, st);
    else if (a.d <= 96) dkv<96>(a, b, st);
    else dkv<128>(a, b, st);
    if (a.rows > ATT_CHECK) {
        if (a.d <= 32) bwd_fine<32>(a, b, st);
        else if (a.d <= 64) bwd_fine<64>(a, b, st);
        else if (a.d <= 96) bwd_fine<96>(a, b, st);
        else bwd_fine<128>(a, b, st);
    }
    prof_end(st, PROF_ATT_DKV);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_attention_round(a, st);
}

}  // namespace ie
