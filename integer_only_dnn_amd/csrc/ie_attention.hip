// Softmax attention over packed sequences, forward.
//
//   t_ij = (q_i . k_j) 2^(e_j),  m_i = max_j t_ij over the keys that i sees,
//   P_ij = rint(w_ij), L_i = sum_j P_ij,  E_i = max e_j over the same keys,
//   P'_ij = rint(w_ij 2^(e_j - E_i)),  o_i = (sum_j P'_ij v_j) 2^(E_i) / L_i
// with w_ij the weight of t_ij - m_i (ie_attn.h).  Sums over keys are exact
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

// A workgroup of four waves takes 128 queries of one head, 32 to a wave, one
// to a lane pair; keys pass through LDS 64 at a time, the next ones in flight.
template <int DP, bool ROW, bool CAUSAL>
__global__ __launch_bounds__(256) void attn_fwd_kernel(AttnArgs p, int slots) {
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
    const int eq = clip_e(xe[ROW ? min(qi, n - 1) : 0]);
    const float r = p.c * pow2f(eq) * (ROW ? 1.0f : pow2f(eq));
    v4i q[NS];
    head_regs<DP>(base + (long long)qi * p.width + h * p.d, ok, p.d, p.vec, lane, q);
    const int keys = CAUSAL ? min(n, q0 + 128) : n, tiles = (keys + 63) / 64;
    const int last = CAUSAL ? min(n, qw + 32) : n;  // keys of this wave
    const bool idle = qw >= n;

    T k, v;
    float fe = 0.0f;
    auto fetch = [&](int t, bool values) {
        k.fetch(kh, p.width, 64 * t, keys, p.d, p.vec);
        if (values) v.fetch(vh, p.width, 64 * t, keys, p.d, p.vec);
        if (ROW && tid < 64) fe = pow2f(clip_e(xe[min(64 * t + tid, n - 1)]));
    };
    auto put = [&](int t, bool values) {
        k.put(sk[t & 1]);
        if (values) v.put(sv[t & 1]);
        if (ROW && tid < 64) sf[t & 1][tid] = fe;
    };
    // scores of 32 keys from key row `at` of a tile
    auto scores = [&](const int8_t *s, int at) {
        v16i acc = {};
#pragma unroll
        for (int i = 0; i < NS; ++i) acc = mfma(T::frag_r(s, at, i, lane), q[i], acc);
        return acc;
    };
    auto sees = [&](int j) { return CAUSAL ? j <= qi : j < n; };
    // whether every key of 32 from j on is seen by every query of the wave
    auto whole = [&](int j) { return j + 32 <= (CAUSAL ? qw + 1 : n); };

    // first pass: the largest score (an int32 where all rows share an exponent)
    float m = -__builtin_inff(), em = 0.0f;
    int mi = -(1 << 30);
    fetch(0, false);
    for (int t = 0; t < tiles; ++t) {
        put(t, false);
        if (t + 1 < tiles) fetch(t + 1, false);
        __syncthreads();
#pragma unroll
        for (int b = 0; b < 64; b += 32) {
            const int j0 = 64 * t + b;
            if (idle || j0 >= last) continue;
            const v16i acc = scores(sk[t & 1], b);
            const bool all = whole(j0);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4 f = ROW ? *(const float4 *)&sf[t & 1][b + 8 * g + 4 * half] : float4{1, 1, 1, 1};
                const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool on = all || sees(j0 + 8 * g + 4 * half + i);
                    if (ROW) {
                        m = fmaxf(m, on ? (float)acc[4 * g + i] * fs[i] : -__builtin_inff());
                        em = fmaxf(em, on ? fs[i] : 0.0f);
                    } else {
                        mi = max(mi, on ? acc[4 * g + i] : -(1 << 30));
                    }
                }
            }
        }
    }
    if (ROW) {
        m = half_max(m);
        em = half_max(em);
    } else {
        mi = swap_reduce<32>(mi, Max{});
    }
    const int top = ROW ? (__float_as_int(em) >> 23) - 127 : eq;  // E
    const float down = ROW ? pow2f(-top) : 1.0f;
    __syncthreads();

    // second pass: weights and the sums they enter
    v16i hi[NS] = {}, lo[NS] = {};
    uint32_t sum = 0;
    fetch(0, true);
    for (int t = 0; t < tiles; ++t) {
        put(t, true);
        if (t + 1 < tiles) fetch(t + 1, true);
        __syncthreads();
#pragma unroll
        for (int b = 0; b < 64; b += 32) {
            const int j0 = 64 * t + b;
            if (idle || j0 >= last) continue;
            const v16i acc = scores(sk[t & 1], b);
            const bool all = whole(j0);
            v4i dh, dl;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float4 f = ROW ? *(const float4 *)&sf[t & 1][b + 8 * g + 4 * half] : float4{1, 1, 1, 1};
                const float fs[4] = {f.x, f.y, f.z, f.w};
                int bits[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float w = ROW ? weight(__builtin_fmaf((float)acc[4 * g + i], fs[i], -m), r)
                                  : weight((float)(acc[4 * g + i] - mi), r);
                    if (!all && !sees(j0 + 8 * g + 4 * half + i)) w = 0.0f;
                    bits[i] = __float_as_int(ROW ? __builtin_fmaf(w, fs[i] * down, RINT_128) : w + RINT_128);
                    sum += ROW ? (uint32_t)__float_as_int(w + RINT_MAGIC) - (uint32_t)RINT_BITS
                               : (uint32_t)bits[i] - (uint32_t)(RINT_BITS + 128);
                }
                int a, c;
                digits4(bits[0], bits[1], bits[2], bits[3], a, c);
                dh[g] = a;
                dl[g] = c;
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const v4i vt = T::frag_t(sv[t & 1], b, s, lane);
                hi[s] = mfma(vt, dh, hi[s]);
                lo[s] = mfma(vt, dl, lo[s]);
            }
        }
    }
    if (idle) return;
    sum = (uint32_t)swap_reduce<32>((int)sum, Add{});
    const double inv = 1.0 / (double)sum;
    double y[16 * NS];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 16; ++i) y[16 * s + i] = __builtin_fma((double)hi[s][i], 256.0, (double)lo[s][i]) * inv;
    const long long row = sp.a + qi;
    store_odd(y, top, p.q, ok, p.d, lane, p.v16 + row * p.cols + h * p.d, p.p16 + row * p.parts + h);
    if (p.stats && ok && lane < 32)
        p.stats[row * p.heads + h] = int2{__float_as_int(ROW ? m : (float)mi * pow2f(eq)), (int)sum};
}

// Rows of heads, each rounded to odd at two bits below its own need, into one
// exponent a row: a wave per row, eight results a lane and turn.
__global__ __launch_bounds__(256) void attn_round_kernel(AttnArgs p) {
    const int lane = threadIdx.x & 63;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= p.rows) return;
    if (p.off && row == 0) {
        bool bad = false;
        for (int s = lane; s < p.n_seq; s += 64) {
            const long long a = p.off[s], b = p.off[s + 1];
            bad |= a < 0 || b < a || b > p.rows || b - a > p.most;
        }
        if (bad) atomicOr(p.flags, IE_FLAG_INDEX);
    }
    if (p.off && (row < p.off[0] || row >= p.off[p.n_seq])) return;  // behind the last sequence: left as it is
    const int16_t *need = p.p16 + row * p.parts;
    int e = P_NONE;
    for (int i = lane; i < p.parts; i += 64) e = max(e, (int)need[i]);
    e = clamp_exp_flag(max(E_MIN, wave_max_dpp(e)), p.flags);
    if (lane == 0) {
        p.ye[row] = (int8_t)e;
        if (p.xe[p.x_row ? row : 0] > ATT_E_HI) atomicOr(p.flags, IE_FLAG_EXP_RANGE);
    }
    const int16_t *v = p.v16 + row * p.cols;
    int8_t *y = p.y + row * p.cols;
    if (p.out_vec) {
        for (int c = 8 * lane; c < p.cols; c += 512) {
            const int s = e - ((int)need[c / p.d] - 2);
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
        for (int c = lane; c < p.cols; c += 64) y[c] = (int8_t)rne_shift32((int)v[c], e - ((int)need[c / p.d] - 2));
    }
}

hipError_t launch_attention_round(const AttnArgs &a, hipStream_t st) {
    prof_begin(st, PROF_ATT_ROUND);
    hipLaunchKernelGGL(attn_round_kernel, dim3((unsigned)((a.rows + 3) / 4)), dim3(256), 0, st, a);
    prof_end(st, PROF_ATT_ROUND);
    return hipGetLastError();
}

template <int DP>
static void fwd(const AttnArgs &a, int slots, dim3 grid, hipStream_t st) {
    const dim3 block(256);
    if (a.x_row) {
        if (a.causal) hipLaunchKernelGGL((attn_fwd_kernel<DP, true, true>), grid, block, 0, st, a, slots);
        else hipLaunchKernelGGL((attn_fwd_kernel<DP, true, false>), grid, block, 0, st, a, slots);
    } else {
        if (a.causal) hipLaunchKernelGGL((attn_fwd_kernel<DP, false, true>), grid, block, 0, st, a, slots);
        else hipLaunchKernelGGL((attn_fwd_kernel<DP, false, false>), grid, block, 0, st, a, slots);
    }
}

hipError_t launch_attention_fwd(const AttnArgs &a, hipStream_t st) {
    const int slots = att_slots(a.rows, a.n_seq, 128);
    const long long total = (long long)slots * a.heads;
    const dim3 grid((unsigned)((total + 7) / 8 * 8));
    prof_begin(st, PROF_ATT_FWD);
    if (a.d <= 32) fwd<32>(a, slots, grid, st);
    else if (a.d <= 64) fwd<64>(a, slots, grid, st);
    else if (a.d <= 96) fwd<96>(a, slots, grid, st);
    else fwd<128>(a, slots, grid, st);
    prof_end(st, PROF_ATT_FWD);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_attention_round(a, st);
}

}  // namespace ie
