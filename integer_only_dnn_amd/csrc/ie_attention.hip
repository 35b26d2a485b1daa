// Softmax attention over packed sequences, forward.
//
//   t_ij = (q_i . k_j) 2^(e_j),  m_i = max_j t_ij over the keys that i sees,
//   P_ij = rint(w_ij), L_i = sum_j P_ij,  E_i = max e_j over the same keys,
//   P'_ij = rint(w_ij 2^(e_j - E_i)),  o_i = (sum_j P'_ij v_j) 2^(E_i) / L_i
// with w_ij the weight of t_ij - m_i (ie_attn.h), in finer units for the rows of
// many small weights.  Sums over keys are exact
// integers, so a row's result depends on the keys it sees alone, and not on
// how they are split into tiles.  The division by L (a product with 1 / L) is
// held to 53 bits; a row's heads are rounded into its one exponent at the end,
// by a second kernel, from round-to-odd values.
//
// Two passes over the keys: the first finds m (and E), the second has the
// final maximum from the start, so that its integers never have to be
// rescaled.  The second product of q and k costs less than rescaling would:
// two matrix instructions and three vector instructions a score beside the
// about fifteen of a weight, its rounding and its digits.
#include "ie_attn.h"

#pragma clang fp contract(off)

namespace ie {

// Rows of nh heads of d elements into heads of dp (a multiple of 16), zeros in
// between: what the kernels read where heads do not start at multiples of 16
// bytes.
__global__ __launch_bounds__(256) void attn_pad_kernel(const int8_t *x, long long rows, int nh, int d, int dp, int8_t *out) {
    const int per = dp >> 4, row_chunks = nh * per;
    const long long n = rows * row_chunks;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const long long row = i / row_chunks;
        const int c = (int)(i - row * row_chunks), h = c / per;
        *(v4i *)(out + i * 16) = head16(x + (row * nh + h) * d, c - h * per, d);
    }
}

hipError_t launch_attention_pad(const int8_t *x, long long rows, int nh, int d, int dp, int8_t *out, hipStream_t st) {
    const long long blocks = (rows * nh * (dp >> 4) + 255) / 256;
    prof_begin(st, PROF_ATT_PAD);
    hipLaunchKernelGGL(attn_pad_kernel, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, st, x, rows, nh, d, dp, out);
    prof_end(st, PROF_ATT_PAD);
    return hipGetLastError();
}

// A workgroup of four waves takes 64 queries of one head, 16 to a wave, one to
// four lanes; keys pass through LDS 64 at a time, the next ones in flight.
//
// SHORT, for batches of short sequences: up to 256 keys have their scores kept
// in registers between the passes (64 of them), so that q and k meet once; all
// keys are in LDS at once, and the values, loaded with them, take their place.
// SPLIT 4: the waves take the same 16 queries and every fourth tile of keys each,
// staged by the wave itself; they share the maximum after the first pass and add
// their sums up after the second.
//
// Bound by vector instructions: 128 x 197 tokens x 12 heads of 64 65 us, 82 % of the
// cycles in which a CU is busy issue one; 5 sequences of 8192 tokens x 32 heads of 128,
// causal, 290 us (142 G operations: 0.49 POP/s), 75 %, and 24 % in matrix instructions.
// Of 29 and 26 instructions to a pair of tokens 15 are the second pass's and 6 the first
// one's, 17 in all where scores are kept; the others are masked keys and queries past a
// sequence's end, the search, and the results' products and rounding in fp64.  Eight waves
// to a workgroup, which halves the loads, waits longer at its barriers (74 and 357 us); 32 x
// 32 products need twice the registers.
template <int DP, bool ROW, bool CAUSAL, bool SHORT, int SPLIT>
__global__ __launch_bounds__(256, SPLIT > 1 ? 2 : DP > 64 ? 3 : 4) void attn_fwd_kernel(AttnArgs p) {
    using T = HeadTile<DP, 256 / SPLIT>;
    constexpr int KS = T::KS, NE = DP / 16, BM = 64 / SPLIT, NB = SPLIT == 1 ? 2 : SPLIT;
    __shared__ __align__(16) int8_t tiles_lds[2 * NB][T::BYTES];
    __shared__ __align__(16) float factors_lds[256];
    __shared__ __align__(16) float scaled_lds[NB][64], most_lds[4];  // factors 2^-E, largest ones
    int8_t(*sk)[T::BYTES] = tiles_lds, (*sv)[T::BYTES] = tiles_lds + NB;
    float(*sf)[64] = (float(*)[64])factors_lds;
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
    const int eq = clip_e(xe[ROW ? min(qi, n - 1) : 0]);
    const float r = p.c * pow2f(eq) * (ROW ? 1.0f : pow2f(eq));
    v4i q[KS];
    head_regs<KS>(base + (long long)qi * p.width + h * p.dp, ok, p.dp, lane, q);
    const int keys = CAUSAL ? min(n, q0 + BM) : n, tiles = (keys + 63) / 64;
    const int last = CAUSAL ? min(n, qw + 16) : n;  // keys of this wave

    v4i hi[NE] = {}, lo[NE] = {};
    uint32_t sum = 0, blocks = 0;
    // the digits of four weights of keys 16 z + 4 quad .., given t - m or the scores' difference, and
    // 2^(e - E): where every query sees every key E is one number, and f has it already
    uint32_t part = 0;  // the weights in units of 2^-7, modulo 2^32
    auto weigh4 = [&](auto masked, auto checked, const float (&d)[4], const float (&f)[4], float down, int z, int lim, int &dh, int &dl) {
        int bits[4];
        uint32_t whole_n[4], seventh[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float w = weight(d[i], r);
            if (masked.value) w = 16 * z + i <= lim ? w : 0.0f;
            bits[i] = __float_as_int(ROW ? __builtin_fmaf(w, CAUSAL ? f[i] * down : f[i], RINT_128) : w + RINT_128);
            whole_n[i] = (uint32_t)(ROW ? __float_as_int(w + RINT_MAGIC) : bits[i]);
            if (checked.value) seventh[i] = (uint32_t)__float_as_int(__builtin_fmaf(w, 128.0f, RINT_MAGIC));
        }
        if (checked.value) {  // modulo 2^32
            part += seventh[0] + seventh[1];
            part += seventh[2] + seventh[3];
        }
        sum += whole_n[0] + whole_n[1];
        sum += whole_n[2] + whole_n[3];
        ++blocks;
        digits4(bits[0], bits[1], bits[2], bits[3], dh, dl);
    };
    auto gather = [&](const int8_t *lds, const v4i &dh, const v4i &dl) {
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const v4i vt = T::frag_t(lds, e, lane);
            hi[e] = mfma(vt, dh, hi[e]);
            lo[e] = mfma(vt, dl, lo[e]);
        }
    };
    auto total = [&]() {
        sum -= 4 * blocks * (uint32_t)(ROW ? RINT_BITS : RINT_BITS + 128);
        sum = (uint32_t)col_reduce((int)sum, Add{});
    };
    // lost: what rounding took of the weights, in units of 2^-7
    auto finish = [&](float m, int mi, int top, int lost = 0) {
        const double inv = 1.0 / (double)sum;
        double y[4 * NE], big = 0.0;
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[4 * e + i] = __builtin_fma((double)hi[e][i], 256.0, (double)lo[e][i]);
        bool fine = false;
        if (keys > ATT_CHECK) {
#pragma unroll
            for (int i = 0; i < 4 * NE; ++i) big = fmax(big, fabs(y[i]));
            big = swap_reduce<32>(swap_reduce<16>(big, MaxD{}), MaxD{});
            const int seen = CAUSAL ? qi + 1 : n;
            fine = ok && seen > ATT_CHECK && (32ll * abs(lost) > 128ll * sum || big < 64.0 * seen);
        }
#pragma unroll
        for (int i = 0; i < 4 * NE; ++i) y[i] *= inv;
        const long long row = sp.a + qi;
        store_odd(y, top, p.q, ok, p.d, lane, p.v16 + row * p.cols + h * p.d, p.p16 + row * p.parts + h);
        if (p.stats && ok && lane < 16)
            p.stats[row * p.heads + h] = int2{__float_as_int(ROW ? m : (float)mi * pow2f(eq)), (int)sum};
        if (fine && lane < 16) {
            p.p16[row * p.parts + h] = P_FINE;
            p.flags[FINE_WORD] = 1;  // the same from every lane that says so
        }
    };

    if constexpr (SHORT) {
        if (n <= 256) {
            T k[4], v[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                k[t].init(p.width, p.dp);
                if (64 * t < keys) k[t].fetch(kh, p.width, 64 * t, keys, p.dp);
            }
            float fe = 0.0f;
            if (ROW) fe = pow2f(clip_e(xe[min(tid, n - 1)]));
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                v[t].init(p.width, p.dp);
                if (64 * t < keys) v[t].fetch(vh, p.width, 64 * t, keys, p.dp);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (64 * t < keys) k[t].put(tiles_lds[t]);
            if (ROW) {
                factors_lds[tid] = fe;
                most_lds[wave] = __int_as_float(wave_max_dpp(__float_as_int(fe)));  // rows behind the last repeat it
            }
            __syncthreads();
            float s[16][4], m = -__builtin_inff(), em = 0.0f;
            int mi = -(1 << 30);
            const int lim = (CAUSAL ? qi : n - 1) - 4 * quad;  // keys 16 z + i <= lim are seen
            auto whole = [&](int t) { return 64 * t + 64 <= (CAUSAL ? qw + 1 : n); };
            auto score = [&](auto masked, int t) {
                constexpr bool each = CAUSAL && decltype(masked)::value;
                if (ROW && !each) em = fmaxf(em, most_lds[t]);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    if (masked.value && 64 * t + 16 * z >= last) continue;
                    v4i acc = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < KS; ++i) acc = mfma(T::frag_r(tiles_lds[t], z, i, lane), q[i], acc);
                    const float4 f = ROW ? *(const float4 *)&factors_lds[64 * t + 16 * z + 4 * quad] : float4{1, 1, 1, 1};
                    const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = (float)acc[i] * fs[i];
                        const bool on = !masked.value || 64 * t + 16 * z + i <= lim;
                        s[4 * t + z][i] = x;
                        m = fmaxf(m, on ? x : -__builtin_inff());
                        if (ROW && each) em = fmaxf(em, on ? fs[i] : 0.0f);
                    }
                }
            };
            auto weigh = [&](auto masked, int t, float down, v4i &dh, v4i &dl) {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    dh[z] = 0;
                    dl[z] = 0;
                    if (masked.value && 64 * t + 16 * z >= last) continue;
                    const float4 x = ROW ? *(const float4 *)&factors_lds[64 * t + 16 * z + 4 * quad] : float4{1, 1, 1, 1};
                    const float f[4] = {x.x, x.y, x.z, x.w};
                    const float(&y)[4] = s[4 * t + z];
                    const float d[4] = {y[0] - m, y[1] - m, y[2] - m, y[3] - m};
                    int a, c;
                    weigh4(masked, Bool<false>{}, d, f, down, 4 * t + z, lim, a, c);
                    dh[z] = a;
                    dl[z] = c;
                }
            };
            if (!idle) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (64 * t < last) {
                        if (whole(t)) score(Bool<false>{}, t);
                        else score(Bool<true>{}, t);
                    }
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (64 * t < keys) v[t].put(tiles_lds[t]);
            if (ROW && !CAUSAL) {
                em = fmaxf(fmaxf(most_lds[0], most_lds[1]), fmaxf(most_lds[2], most_lds[3]));
                factors_lds[tid] = fe * __int_as_float((254 << 23) - __float_as_int(em));
            }
            __syncthreads();
            if (idle) return;
            m = col_max(m);
            if (CAUSAL) em = col_max(em);
            const int top = ROW ? (__float_as_int(em) >> 23) - 127 : eq;
            const float down = ROW ? pow2f(-top) : 1.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (64 * t >= last) break;
                v4i dh, dl;
                if (whole(t)) weigh(Bool<false>{}, t, down, dh, dl);
                else weigh(Bool<true>{}, t, down, dh, dl);
                gather(tiles_lds[t], dh, dl);
            }
            mi = (int)m;  // where all rows share an exponent the scores are whole
            total();
            finish(m, mi, top);
            return;
        }
    }

    T k, v;
    k.init(p.width, p.dp);
    v.init(p.width, p.dp);
    float fe = 0.0f, down = 1.0f;
    // SPLIT: a wave takes every fourth tile, and stages it itself
    const int me = SPLIT == 1 ? tid : lane, first = SPLIT == 1 ? 0 : wave;
    auto buffer = [&](int t) { return SPLIT == 1 ? t & 1 : wave; };
    auto fence = [&]() {
        if (SPLIT == 1) __syncthreads();
        else __builtin_amdgcn_wave_barrier();
    };
    auto fetch = [&](int t, bool values) {
        k.fetch(kh, p.width, 64 * t, keys, p.dp);
        if (values) v.fetch(vh, p.width, 64 * t, keys, p.dp);
        if (ROW && me < 64) fe = pow2f(clip_e(xe[min(64 * t + me, n - 1)]));
    };
    auto put = [&](int t, bool values) {
        if (SPLIT > 1) __builtin_amdgcn_wave_barrier();
        k.put(sk[buffer(t)]);
        if (values) v.put(sv[buffer(t)]);
        if (ROW && me < 64) {
            sf[buffer(t)][me] = fe;
            if (!CAUSAL && values) scaled_lds[buffer(t)][me] = fe * down;
            if (!values) most_lds[buffer(t)] = __int_as_float(wave_max_dpp(__float_as_int(fe)));
        }
    };
    // scores of 16 keys of a tile
    auto scores = [&](int t, int z) {
        v4i acc = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < KS; ++i) acc = mfma(T::frag_r(sk[buffer(t)], z, i, lane), q[i], acc);
        return acc;
    };
    auto factors = [&](const float *at, int z, float (&f)[4]) {
        const float4 x = ROW ? *(const float4 *)(at + 16 * z + 4 * quad) : float4{1, 1, 1, 1};
        f[0] = x.x;
        f[1] = x.y;
        f[2] = x.z;
        f[3] = x.w;
    };
    // whether every key of a tile is seen by every query of the wave; else keys 16 z + i <= limit are seen
    auto whole = [&](int t) { return 64 * t + 64 <= (CAUSAL ? qw + 1 : n); };
    auto limit = [&](int t) { return (CAUSAL ? qi : n - 1) - 64 * t - 4 * quad; };

    // first pass: the largest score (an int32 where all rows share an exponent)
    float m = -__builtin_inff(), em = 0.0f;
    int mi = -(1 << 30);
    auto largest = [&](auto masked, int t) {
        constexpr bool each = CAUSAL && decltype(masked)::value;
        const int lim = limit(t);
        if (ROW && !each) em = fmaxf(em, most_lds[buffer(t)]);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            if (masked.value && 64 * t + 16 * z >= last) break;
            const v4i acc = scores(t, z);
            float f[4];
            factors(sf[buffer(t)], z, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool on = !masked.value || 16 * z + i <= lim;
                if (ROW) {
                    m = fmaxf(m, on ? (float)acc[i] * f[i] : -__builtin_inff());
                    if (each) em = fmaxf(em, on ? f[i] : 0.0f);
                } else {
                    mi = max(mi, on ? acc[i] : -(1 << 30));
                }
            }
        }
    };
    if (first < tiles) fetch(first, false);
    for (int t = first; t < tiles; t += SPLIT) {
        put(t, false);
        if (t + SPLIT < tiles) fetch(t + SPLIT, false);
        fence();
        if (idle) continue;
        if (whole(t)) largest(Bool<false>{}, t);
        else largest(Bool<true>{}, t);
    }
    if (ROW) {
        m = col_max(m);
        if (CAUSAL) em = col_max(em);
    } else {
        mi = col_reduce(mi, Max{});
    }
    if constexpr (SPLIT > 1) {
        __shared__ float sm[2][4][16];
        __shared__ int smi[4][16];
        if (lane < 16) {
            sm[0][wave][lane] = m;
            sm[1][wave][lane] = em;
            smi[wave][lane] = mi;
        }
        __syncthreads();
        const int col = lane & 15;
        m = fmaxf(fmaxf(sm[0][0][col], sm[0][1][col]), fmaxf(sm[0][2][col], sm[0][3][col]));
        em = fmaxf(fmaxf(sm[1][0][col], sm[1][1][col]), fmaxf(sm[1][2][col], sm[1][3][col]));
        mi = max(max(smi[0][col], smi[1][col]), max(smi[2][col], smi[3][col]));
    }
    const int top = ROW ? (__float_as_int(em) >> 23) - 127 : eq;  // E
    if (ROW) down = pow2f(-top);
    __syncthreads();

    // second pass: weights and the sums they enter
    auto weigh = [&](auto masked, auto checked, int t, v4i &dh, v4i &dl) {
        const int lim = limit(t);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            dh[z] = 0;
            dl[z] = 0;
            if (masked.value && 64 * t + 16 * z >= last) continue;
            const v4i acc = scores(t, z);
            float f[4], d[4];
            factors(sf[buffer(t)], z, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = ROW ? __builtin_fmaf((float)acc[i], f[i], -m) : (float)(acc[i] - mi);
            int a, c;
            if (!CAUSAL) factors(scaled_lds[buffer(t)], z, f);
            weigh4(masked, checked, d, f, down, z, lim, a, c);
            dh[z] = a;
            dl[z] = c;
        }
    };
    auto weigh_all = [&](auto checked) {
        if (first < tiles) fetch(first, true);
        for (int t = first; t < tiles; t += SPLIT) {
            put(t, true);
            if (t + SPLIT < tiles) fetch(t + SPLIT, true);
            fence();
            if (idle || 64 * t >= last) continue;
            v4i dh, dl;
            if (whole(t)) weigh(Bool<false>{}, checked, t, dh, dl);
            else weigh(Bool<true>{}, checked, t, dh, dl);
            gather(sv[buffer(t)], dh, dl);
        }
    };
    const bool check = keys > ATT_CHECK;  // rows may need fine weights
    if (check) weigh_all(Bool<true>{});
    else weigh_all(Bool<false>{});
    int lost = 0;
    if (check) {
        const uint32_t n4 = 4 * blocks;
        lost = (int)(part - n4 * (uint32_t)RINT_BITS - 128 * (sum - n4 * (uint32_t)(ROW ? RINT_BITS : RINT_BITS + 128)));
        lost = col_reduce(lost, Add{});
    }
    total();
    if constexpr (SPLIT > 1) {
        int *x = (int *)&tiles_lds[0][0];
        static_assert(sizeof tiles_lds >= 3 * 4 * NE * 64 * sizeof(int), "a digit's sums fit the tiles");
        gather_waves<4 * NE>(x, hi, wave, lane);
        gather_waves<4 * NE>(x, lo, wave, lane);
        v4i s4 = {(int)sum, lost, 0, 0};
        gather_waves<4>(x, (v4i(&)[1])s4, wave, lane);
        sum = (uint32_t)s4[0];
        lost = s4[1];
        if (wave) return;
    }
    if (!idle) finish(m, mi, top, lost);
}

// The rows that the kernel above has marked, with fine weights: the same tiles,
// the sums in four digits.  Launched where a sequence may be long enough for such a
// row; a call without one ends at its first load.  With them in the kernel above,
// behind its sums, its registers ran over (8192 tokens, heads of 128: 667 us for 290).
template <int DP, bool ROW, bool CAUSAL>
__global__ __launch_bounds__(256, DP > 64 ? 1 : 2) void attn_fwd_fine_kernel(AttnArgs p, int items) {
    using T = HeadTile<DP>;
    constexpr int KS = T::KS, NE = DP / 16;
    __shared__ __align__(16) int8_t sk[2][T::BYTES], sv[2][T::BYTES];
    __shared__ __align__(16) float sf[2][64];
    __shared__ int any_lds[4];
    if (!p.flags[FINE_WORD]) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, quad = lane >> 4;
    T k, v;
    k.init(p.width, p.dp);
    v.init(p.width, p.dp);
    for (int idx = blockIdx.x; idx < items; idx += gridDim.x) {
        const Item it = att_item(p, p.group, idx, items);
        const int kvh = it.kvh, h = kvh * p.group + it.gh;
        Span sp;
        int tile;
        if (!rank_tile<CAUSAL>(p, it.rank, 64, sp, tile)) continue;
        const int n = sp.n, q0 = 64 * tile, qw = q0 + 16 * wave, qi = qw + (lane & 15);
        const long long row = sp.a + qi;
        const bool fine = qi < n && p.p16[row * p.parts + h] == P_FINE;
        const bool some = __ballot(fine) != 0;
        __syncthreads();  // the tiles before are read
        if (lane == 0) any_lds[wave] = some;
        __syncthreads();
        if (!(any_lds[0] | any_lds[1] | any_lds[2] | any_lds[3])) continue;
        const int8_t *base = p.x + (long long)sp.a * p.width;
        const int8_t *kh = base + (long long)(p.heads + kvh) * p.dp, *vh = kh + (long long)p.kv * p.dp;
        const int8_t *xe = p.xe + (ROW ? sp.a : 0);
        const int eq = clip_e(xe[ROW ? min(qi, n - 1) : 0]);
        const float r = p.c * pow2f(eq) * (ROW ? 1.0f : pow2f(eq));
        v4i q[KS];
        head_regs<KS>(base + (long long)qi * p.width + h * p.dp, qi < n, p.dp, lane, q);
        const int keys = CAUSAL ? min(n, q0 + 64) : n, tiles = (keys + 63) / 64, lim = CAUSAL ? qi : n - 1;
        float fe = 0.0f;
        auto fetch = [&](int t, bool values) {
            k.fetch(kh, p.width, 64 * t, keys, p.dp);
            if (values) v.fetch(vh, p.width, 64 * t, keys, p.dp);
            if (tid < 64) fe = ROW ? pow2f(clip_e(xe[min(64 * t + tid, n - 1)])) : 1.0f;
        };
        auto put = [&](int t, bool values) {
            k.put(sk[t & 1]);
            if (values) v.put(sv[t & 1]);
            if (tid < 64) sf[t & 1][tid] = fe;
        };
        auto scores = [&](int t, int z) {
            v4i acc = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KS; ++i) acc = mfma(T::frag_r(sk[t & 1], z, i, lane), q[i], acc);
            return acc;
        };
        // the largest score, and the largest factor of the keys seen
        float m = -__builtin_inff(), em = 0.0f;
        fetch(0, false);
        for (int t = 0; t < tiles; ++t) {
            put(t, false);
            if (t + 1 < tiles) fetch(t + 1, false);
            __syncthreads();
            if (!some) continue;
            for (int z = 0; z < 4; ++z) {
                const v4i acc = scores(t, z);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool on = 64 * t + 16 * z + 4 * quad + i <= lim;
                    const float f = sf[t & 1][16 * z + 4 * quad + i];
                    m = fmaxf(m, on ? (float)acc[i] * f : -__builtin_inff());
                    em = fmaxf(em, on ? f : 0.0f);
                }
            }
        }
        m = col_max(m);
        em = col_max(em);
        const int top = ROW ? (__float_as_int(em) >> 23) - 127 : eq;
        const float down = pow2f(ROW ? -top : 0);
        __syncthreads();
        v4i acc[4][NE] = {};
        long long count = 0;
        fetch(0, true);
        for (int t = 0; t < tiles; ++t) {
            put(t, true);
            if (t + 1 < tiles) fetch(t + 1, true);
            __syncthreads();
            if (!some) continue;
            v4i dg[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const v4i s = scores(t, z);
                int n4[4], o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = sf[t & 1][16 * z + 4 * quad + i];
                    float w = weight(__builtin_fmaf((float)s[i], f, -m), r);
                    w = 64 * t + 16 * z + 4 * quad + i <= lim ? w : 0.0f;
                    count += (int)__builtin_rintf(w * FINE_UNIT);
                    n4[i] = (int)__builtin_rintf(w * (ROW ? f * down : 1.0f) * FINE_UNIT);
                }
                digits4x4(n4, o);
#pragma unroll
                for (int g = 0; g < 4; ++g) dg[g][z] = o[g];
            }
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                const v4i vt = T::frag_t(sv[t & 1], e, lane);
#pragma unroll
                for (int g = 0; g < 4; ++g) acc[g][e] = mfma(vt, dg[g], acc[g][e]);
            }
        }
        if (!some) continue;
        const double total = swap_reduce<32>(swap_reduce<16>((double)count, Add{}), Add{}), inv = 1.0 / total;
        double y[4 * NE];
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[4 * e + i] = whole4(acc[0][e][i], acc[1][e][i], acc[2][e][i], acc[3][e][i]) * inv;
        store_odd(y, top, p.q, fine, p.d, lane, p.v16 + row * p.cols + h * p.d, p.p16 + row * p.parts + h);
        if (p.stats && fine && lane < 16)
            p.stats[row * p.heads + h] = int2{__float_as_int(ROW ? m : m * pow2f(eq)) | 1, (int)(uint32_t)rint(total * (1.0 / 16384.0))};
    }
}

// Rows of parts (heads), each rounded to odd at two bits below its own need, into one
// exponent a row: T threads per row (a wave, or a workgroup for few rows: 48 rows of
// 4096 4.1 us and with waves 7.4; 25216 of 768 28 and 15), eight results a thread and
// turn.  A stream: 25216 rows of 2304 (174 MB) 30 us.
template <int T>
__global__ __launch_bounds__(256) void attn_round_kernel(AttnArgs p) {
    __shared__ int sh[4];
    const int lane = threadIdx.x % T;
    const long long row = (long long)blockIdx.x * (256 / T) + threadIdx.x / T;
    if (row >= p.rows) return;
    if (row == 0 && lane == 0) p.flags[FINE_WORD] = 0;
    if (p.off && row == 0) {
        bool bad = false;
        for (int s = lane; s < p.n_seq; s += T) {
            const long long a = p.off[s], b = p.off[s + 1];
            bad |= a < 0 || b < a || b > p.rows || b - a > p.most;
        }
        if (bad) atomicOr(p.flags, IE_FLAG_INDEX);
    }
    if (p.off && (row < p.off[0] || row >= p.off[p.n_seq])) return;  // behind the last sequence: left as it is
    const int16_t *need = p.p16 + row * p.parts;
    int e = P_NONE;
    for (int i = lane; i < p.parts; i += T) e = max(e, (int)need[i]);
    e = clamp_exp_flag(max(E_MIN, row_reduce<T>(e, Max{}, sh)), p.flags);
    if (lane == 0) {
        p.ye[row] = (int8_t)e;
        if (p.xe[p.x_row ? row : 0] > ATT_E_HI) atomicOr(p.flags, IE_FLAG_EXP_RANGE);
    }
    const int16_t *v = p.v16 + row * p.cols;
    int8_t *y = p.y + row * p.cols;
    if (p.out_vec) {
        for (int c = 8 * lane; c < p.cols; c += 8 * T) {
            const int s = e - ((int)need[c / p.part] - 2);
            const v4i w = *(const v4i *)(v + c);
            int o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o[2 * k] = rne_shift32((int)(int16_t)w[k], s);
                o[2 * k + 1] = rne_shift32(w[k] >> 16, s);
            }
            *(uint2 *)(y + c) = uint2{pack4(o[0], o[1], o[2], o[3]), pack4(o[4], o[5], o[6], o[7])};
        }
    } else {
        for (int c = lane; c < p.cols; c += T) y[c] = (int8_t)rne_shift32((int)v[c], e - ((int)need[c / p.part] - 2));
    }
}

hipError_t launch_attention_round(const AttnArgs &a, hipStream_t st) {
    prof_begin(st, PROF_ATT_ROUND);
    if (a.rows < 4 * NCU) hipLaunchKernelGGL(attn_round_kernel<256>, dim3((unsigned)a.rows), dim3(256), 0, st, a);
    else hipLaunchKernelGGL(attn_round_kernel<64>, dim3((unsigned)((a.rows + 3) / 4)), dim3(256), 0, st, a);
    prof_end(st, PROF_ATT_ROUND);
    return hipGetLastError();
}

template <int DP>
static void fwd_fine(const AttnArgs &a, hipStream_t st) {
    const unsigned items = att_grid(att_slots(a.rows, a.n_seq, 64), a.kv, a.group);
    const dim3 grid(items < 2 * NCU ? items : 2 * NCU), block(256);
    if (a.x_row) {
        if (a.causal) hipLaunchKernelGGL((attn_fwd_fine_kernel<DP, true, true>), grid, block, 0, st, a, (int)items);
        else hipLaunchKernelGGL((attn_fwd_fine_kernel<DP, true, false>), grid, block, 0, st, a, (int)items);
    } else {
        if (a.causal) hipLaunchKernelGGL((attn_fwd_fine_kernel<DP, false, true>), grid, block, 0, st, a, (int)items);
        else hipLaunchKernelGGL((attn_fwd_fine_kernel<DP, false, false>), grid, block, 0, st, a, (int)items);
    }
}

template <int DP, bool SHORT, int SPLIT>
static void fwd(AttnArgs a, hipStream_t st) {
    a.chunk = att_chunk(a, 64 / SPLIT, !a.causal);
    const dim3 grid(att_grid(att_slots(a.rows, a.n_seq, 64 / SPLIT), a.kv, a.group)), block(256);
    if (a.x_row) {
        if (a.causal) hipLaunchKernelGGL((attn_fwd_kernel<DP, true, true, SHORT, SPLIT>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((attn_fwd_kernel<DP, true, false, SHORT, SPLIT>), grid, block, 0, st, a);
    } else {
        if (a.causal) hipLaunchKernelGGL((attn_fwd_kernel<DP, false, true, SHORT, SPLIT>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((attn_fwd_kernel<DP, false, false, SHORT, SPLIT>), grid, block, 0, st, a);
    }
}

template <int DP>
static void fwd(const AttnArgs &a, hipStream_t st) {
    // sequences of up to 256 tokens on the average: most have their scores in registers (128 x
    // 197 x 12 heads of 64: 68 us, with two products 83; longer sequences lose 1 % in that kernel).
    // Fewer tiles than two a CU: split (tokens x heads of 64, causal, split and whole: 1024 x 8 14
    // and 27 us, 2048 x 8 29 and 50; 1024 x 16, all keys seen, 27 and 31)
    if (a.rows <= 256ll * max(a.n_seq, 1)) fwd<DP, true, 1>(a, st);
    else if (att_slots(a.rows, a.n_seq, 64) * a.heads < 2 * NCU) fwd<DP, false, 4>(a, st);
    else fwd<DP, false, 1>(a, st);
    if (a.rows > ATT_CHECK) fwd_fine<DP>(a, st);
}

hipError_t launch_attention_fwd(const AttnArgs &a, hipStream_t st) {
    prof_begin(st, PROF_ATT_FWD);
    if (a.d <= 32) fwd<32>(a, st);
    else if (a.d <= 64) fwd<64>(a, st);
    else if (a.d <= 96) fwd<96>(a, st);
    else fwd<128>(a, st);
    prof_end(st, PROF_ATT_FWD);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_attention_round(a, st);
}

}  // namespace ie
