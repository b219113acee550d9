// Attention over jagged sequences, backward (dlrm_seq.h).
//
//   P = exp(z - lse);  dP = dO V^T;  ds = P (dP - <dO, o>)
//   dQ = scale ds K;  dK = scale ds^T Q;  dV = P^T dO;  dbias[t] = sum of ds over bucket t
//
// P is computed again from Q, K and the saved log-sums.  Two kernels, so that every sum has an owner
// and no gradient is added to by atomics: one over blocks of queries (dQ, dbias and <dO, o>), one
// over blocks of keys (dK, dV; it walks the query heads that share the key head one after the
// other).  That computes S and dP twice: 7 products of Q x K x d instead of the 5 that one kernel
// with atomic dQ would need.  Both work on the tiles of the forward: the accumulator of S and dP
// becomes the next product's operand in registers, and the transposed operands (K^T; Q^T and dO^T)
// are read from row-major tiles by transposing LDS loads.
#include <type_traits>

#include "seq.h"

namespace dlrm {
namespace seq {
namespace {

// Rows of one slot table of partial bias gradients: [head][slot][bucket].
struct Grads {
    const uint16_t *dout, *o;
    const float *o_lo, *lse;
    float *delta;    // [Nq][Hq]
    float *partial;  // [Hq][slots][buckets]
    uint16_t *dq, *dk, *dv;
};

template <int CTRL, int ROWS>
__device__ __forceinline__ void segment_step(float &x, int t) {
    const float up = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, false));
    const int tup = __builtin_amdgcn_update_dpp(-1, t, CTRL, ROWS, 0xf, false);
    x += tup == t ? up : 0.f;
}

// Adds each lane's x to sums[t] (one wavefront's own array in LDS); t does not decrease over the
// lanes.  A scan within equal t, then the last lane of each writes: no atomics, one fixed order.
__device__ __forceinline__ void add_by_bucket(float *sums, float x, int t, int lane) {
    segment_step<0x111, 0xf>(x, t);  // row_shr:1, 2, 4, 8 within 16 lanes
    segment_step<0x112, 0xf>(x, t);
    segment_step<0x114, 0xf>(x, t);
    segment_step<0x118, 0xf>(x, t);
    segment_step<0x142, 0xa>(x, t);  // row_bcast:15 into rows 1 and 3
    segment_step<0x143, 0xc>(x, t);  // row_bcast:31 into rows 2 and 3
    const int next = __shfl_down(t, 1);
    if (lane == 63 || next != t) sums[t] += x;
    wave_lds_sync();
}

template <int DP, int LP, int NW>
__global__ __launch_bounds__(NW * 64) void k_seq_attn_bwd_q(const Args a, const Grads gr, const int64_t slots) {
    constexpr int QT = NW * 32, STEPS = DP / 16, MB = DP / 32, THREADS = NW * 64;
    constexpr int TAB = QT + kBK, PITCH = 36;
    __shared__ __attribute__((aligned(16))) uint16_t Ks[2][kBK * LP], Vs[2][kBK * LP];
    __shared__ __attribute__((aligned(16))) float skew[NW][32 * PITCH];
    __shared__ float tab[2][TAB], bias_s[DLRM_SEQ_MAX_BUCKETS], sums[NW][DLRM_SEQ_MAX_BUCKETS];
    __shared__ int bounds_s[DLRM_SEQ_MAX_BUCKETS];
    __shared__ uint8_t btab[2][TAB];

    const int64_t id = xcd_contiguous(blockIdx.x, gridDim.x);
    if (id >= slots * a.Hq) return;
    const int h = static_cast<int>(id / slots);
    const int64_t slot = id - h * slots;
    const int b = find_sequence(a, a.q_off, a.Nq, slot, QT);
    const Span sp = span_of(a, b);
    const int64_t t = slot - (sp.q0 / QT + b);
    const int tiles = (sp.qlen + QT - 1) / QT;
    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, half = lane >> 5;
    if (t < 0 || t >= tiles) {
        for (int i = tid; i < a.buckets; i += THREADS) gr.partial[id * a.buckets + i] = 0.f;
        return;
    }
    const int q0 = (tiles - 1 - static_cast<int>(t)) * QT;
    const int w = static_cast<int>(wave_id());
    const int kvh = h / a.group;
    const uint16_t *kb = a.k + sp.k0 * a.k_row + kvh * a.k_head;
    const uint16_t *vb = a.v + sp.k0 * a.v_row + kvh * a.v_head;

    for (int i = tid; i < a.buckets; i += THREADS) {
        bounds_s[i] = a.bounds[i];
        bias_s[i] = a.bias[static_cast<int64_t>(h) * a.buckets + i];
    }
    const int ql = q0 + w * 32 + ln;
    const bool live = ql < sp.qlen;
    const int64_t orow = ((sp.q0 + ql) * a.Hq + h) * static_cast<int64_t>(a.d);
    Frag qf[STEPS], df[STEPS];
    float delta = 0.f, lse = kInf;  // a query that sees nothing: P = exp(z - infinity) = 0
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        qf[s].q = df[s].q = u32x4{0, 0, 0, 0};
        const int c = 16 * s + 8 * half;
        if (live && c < a.d) {
            qf[s].q = *(const DLRM_GLOBAL u32x4 *)(a.q + (sp.q0 + ql) * a.q_row + h * a.q_head + c);
            df[s].q = *(const DLRM_GLOBAL u32x4 *)(gr.dout + orow + c);
            const u32x4 hi = *(const DLRM_GLOBAL u32x4 *)(gr.o + orow + c);
            uint32_t lo[8];
            gload_words<8>(gr.o_lo + orow + c, lo);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                delta = fmaf(bf16_lo(df[s].w[e]), bf16_lo(hi[e]) + __uint_as_float(lo[2 * e]), delta);
                delta = fmaf(bf16_hi(df[s].w[e]), bf16_hi(hi[e]) + __uint_as_float(lo[2 * e + 1]), delta);
            }
        }
    }
    delta = add_halves(delta);
    if (live) {
        const float x = gr.lse[(sp.q0 + ql) * a.Hq + h];
        if (x != -kInf) lse = x;
        if (half == 0) gr.delta[(sp.q0 + ql) * a.Hq + h] = delta;
    }
    const bool huge = __any(fabsf(lse) > kHuge && fabsf(lse) < kInf);
    const float lse2 = lse * kLog2e;

    const int pmin = q0 + sp.shift, pmax = min(q0 + QT, sp.qlen) - 1 + sp.shift;
    const int end = min(sp.klen, pmax + 1);
    const int first = a.window ? max(0, pmin - a.window + 1) : 0;
    const int t1 = end > 0 ? (end + kBK - 1) / kBK : 0;
    const int t0 = min(first / kBK, t1);
    const int nsink = min((a.sinks + kBK - 1) / kBK, t0);
    const int n = nsink + t1 - t0;

    Stage<LP, THREADS> ks, vs;
    const auto key0 = [&](int it) { return (it < nsink ? it : t0 + it - nsink) * kBK; };
    const auto load = [&](int it) {
        ks.load(kb, a.k_row, a.d, key0(it), first, end, a.sinks);
        vs.load(vb, a.v_row, a.d, key0(it), first, end, a.sinks);
    };
    const auto whole = [&](int k0) {
        return pmin - (k0 + kBK - 1) >= 0 && (!a.window || q0 + QT - 1 + sp.shift - k0 < a.window || k0 + kBK <= a.sinks);
    };
    const auto even = [&](int k0) { return whole(k0) && pmin - (k0 + kBK - 1) >= a.last; };
    const auto fill = [&](int it) {
        const int k0 = key0(it), buf = it & 1;
        ks.store(Ks[buf]);
        vs.store(Vs[buf]);
        if (!even(k0)) {
            const int n0 = pmin - (k0 + kBK - 1);
            for (int i = tid; i < TAB - 1; i += THREADS) {
                int bucket;
                tab[buf][i] = table_entry(a, bounds_s, bias_s, n0 + i, k0 < a.sinks, &bucket);
                btab[buf][i] = static_cast<uint8_t>(bucket);
            }
        }
    };

    f32x16 dq[MB];
    float far = 0.f;           // ds summed over the pairs of the last bucket, where a tile has only those
    float carry = 0.f;         // see below
    int carry_key = -1;        // the tile that it goes on in
    const auto drop_carry = [&] {  // distances pmin + 32 w - carry_key + ln
        if (carry_key < 0) return;
        const int dist = pmin + 32 * w - carry_key + ln;
        const float x = add_halves(carry);
        const int bt = half ? a.buckets - 1 : bucket_of(bounds_s, a.buckets, max(dist, 0));
        add_by_bucket(sums[w], half ? 0.f : x, bt, lane);
        carry = 0.f, carry_key = -1;
    };

    const auto pass = [&](auto is_wild) {  // WILD: a second pass, as in the forward
    constexpr bool WILD = decltype(is_wild)::value;
#pragma unroll
    for (int m = 0; m < MB; ++m) dq[m] = f32x16{};
    far = carry = 0.f, carry_key = -1;
    for (int i = tid; i < NW * DLRM_SEQ_MAX_BUCKETS; i += THREADS) sums[0][i] = 0.f;
    if (n > 0) load(0);
    __syncthreads();
    if (n > 0) fill(0);
    for (int it = 0; it < n; ++it) {
        const int k0 = key0(it), buf = it & 1;
        if (it + 1 < n) load(it + 1);
        __syncthreads();
        const int wpos = pmin + w * 32;
        const bool none = wpos + 31 < k0 || q0 + w * 32 >= sp.qlen ||
                          (a.window && wpos - (k0 + kBK - 1) >= a.window && k0 >= a.sinks);
        if (!none) {
            const bool flat = even(k0);
            const bool near = a.buckets && !flat;
            float hi[2], lo[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    Frag k, v;
                    read_row<LP>(k, Ks[buf], 32 * g + ln, 2 * i + half);
                    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k.b, qf[i].b, s, 0, 0, 0);
                    read_row<LP>(v, Vs[buf], 32 * g + ln, 2 * i + half);
                    dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, df[i].b, dp, 0, 0, 0);
                }
                if (flat) {
                    const float c = a.buckets ? bias_s[a.buckets - 1] : 0.f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, c);
                } else {
                    const float *tb = tab[buf] + w * 32 + ln + kBK - 1 - 4 * half - 32 * g;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, tb[-(8 * (r / 4) + r % 4)]);
                    if constexpr (WILD) {
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (tb[-(8 * (r / 4) + r % 4)] == -kInf) s[r] = -kInf;
                    }
                    if (k0 < a.sinks) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int key = k0 + 32 * g + 8 * (r / 4) + 4 * half + r % 4;
                            if (wpos + ln - key >= a.window && key >= a.sinks) s[r] = -kInf;
                        }
                    }
                }
                if (huge) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f((s[r] - lse) * kLog2e);
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], kLog2e, -lse2));
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) dp[r] = s[r] * (dp[r] - delta);
                if constexpr (WILD) {  // a hidden key's dP may be NaN
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (s[r] == 0.f) dp[r] = 0.f;
                }
                Frag ds[2];
#pragma unroll
                for (int r = 0; r < 16; r += 2) ds[r / 8].w[r / 2 % 4] = pack_bf16(dp[r], dp[r + 1]);
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        Frag k;
                        read_columns<LP>(k, Ks[buf], 32 * g + 16 * u, 32 * m, lane);
                        if constexpr (WILD) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) k.w[e] = only_finite(k.w[e]);
                        }
                        dq[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k.b, ds[u].b, dq[m], 0, 0, 0);
                    }
                if (!a.buckets) continue;
                if (flat) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) far += dp[r];
                } else {
                    // the block's sums along its diagonals: through LDS as rows of queries, of which
                    // lane ln then takes key q - ln (mod 32) of query q.  Those with q >= ln are at
                    // distance D + ln, the others at D + ln - 32, D = wpos - k0 - 32 g.
                    float *sk = skew[w];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<floatx4 *>(sk + ln * PITCH + 8 * j + 4 * half) =
                            floatx4{dp[4 * j], dp[4 * j + 1], dp[4 * j + 2], dp[4 * j + 3]};
                    wave_lds_sync();
                    hi[g] = lo[g] = 0.f;
                    const int edge = ln - 16 * half;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int q = 16 * half + i;
                        const float x = sk[q * PITCH + ((q - ln) & 31)];
                        hi[g] += i >= edge ? x : 0.f;
                        lo[g] += i >= edge ? 0.f : x;
                    }
                    wave_lds_sync();
                }
            }
            if (near) {
                // distances of the two blocks' sums, with D = wpos - k0: hi[0] D + ln; lo[0] and hi[1]
                // D + ln - 32; lo[1] D + ln - 64, which is hi[0]'s place in the next tile
                if (carry_key != k0) drop_carry();
                const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(lo[0] + hi[1]),
                                                                __float_as_uint(carry + hi[0]), false, false);
                const float x = __uint_as_float(r[0]) + __uint_as_float(r[1]);  // distance D - 32 + lane
                add_by_bucket(sums[w], x, btab[buf][w * 32 + 31 + lane], lane);
                carry = lo[1], carry_key = k0 + kBK;
            }
        }
        if (it + 1 < n) fill(it + 1);
    }
    };
    pass(std::false_type());
    float any = 0.f;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) any += dq[m][r];
    if (__syncthreads_or(any != any)) pass(std::true_type());
    if (a.buckets) {
        drop_carry();
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) far += __shfl_xor(far, i);
        if (lane == 0) sums[w][a.buckets - 1] += far;
        __syncthreads();
        for (int i = tid; i < a.buckets; i += THREADS) {
            float x = 0.f;
#pragma unroll
            for (int v = 0; v < NW; ++v) x += sums[v][i];
            gr.partial[id * a.buckets + i] = x;
        }
    }
    if (!live) return;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * m + 8 * g + 4 * half;
            if (c >= a.d) continue;
            *(DLRM_GLOBAL u32x2 *)(gr.dq + orow + c) =
                u32x2{pack_bf16(dq[m][4 * g] * a.scale, dq[m][4 * g + 1] * a.scale),
                      pack_bf16(dq[m][4 * g + 2] * a.scale, dq[m][4 * g + 3] * a.scale)};
        }
}

template <int DP, int LP, int NW>
__global__ __launch_bounds__(NW * 64) void k_seq_attn_bwd_kv(const Args a, const Grads gr, const int64_t slots) {
    constexpr int KT = NW * 32, STEPS = DP / 16, MB = DP / 32, THREADS = NW * 64;
    constexpr int TAB = KT + kBK;
    __shared__ __attribute__((aligned(16))) uint16_t Qs[2][kBK * LP], Ds[2][kBK * LP];
    __shared__ __attribute__((aligned(16))) float lse_s[2][kBK], delta_s[2][kBK];
    __shared__ float tab[2][TAB], bias_s[DLRM_SEQ_MAX_BUCKETS];
    __shared__ int bounds_s[DLRM_SEQ_MAX_BUCKETS], huge_s[2];

    const int64_t id = xcd_contiguous(blockIdx.x, gridDim.x);
    if (id >= slots * a.Hkv) return;
    const int kvh = static_cast<int>(id / slots);
    const int64_t slot = id - kvh * slots;
    const int b = find_sequence(a, a.kv_begin, a.Nkv, slot, KT);
    const Span sp = span_of(a, b);
    const int64_t t = slot - (sp.k0 / KT + b);
    const int tiles = (sp.klen + KT - 1) / KT;
    if (t < 0 || t >= tiles) return;
    const int k0 = static_cast<int>(t) * KT;  // the first keys are seen by the most queries: first

    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, half = lane >> 5;
    const int w = static_cast<int>(wave_id());
    const int kl = k0 + w * 32 + ln;
    const bool live = kl < sp.klen;
    Frag kf[STEPS], vf[STEPS];
    bool odd = false;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        kf[s].q = vf[s].q = u32x4{0, 0, 0, 0};
        const int c = 16 * s + 8 * half;
        if (live && c < a.d) {
            kf[s].q = *(const DLRM_GLOBAL u32x4 *)(a.k + (sp.k0 + kl) * a.k_row + kvh * a.k_head + c);
            vf[s].q = *(const DLRM_GLOBAL u32x4 *)(a.v + (sp.k0 + kl) * a.v_row + kvh * a.v_head + c);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            odd |= only_finite(kf[s].w[e]) != kf[s].w[e] || only_finite(vf[s].w[e]) != vf[s].w[e];
    }
    const bool wild = __any(odd);  // a hidden key that is not finite keeps its gradients of zero

    // the queries that see one of the block's keys
    const int qlo = max(0, k0 - sp.shift);
    const int64_t reach = static_cast<int64_t>(k0) + KT - 1 + a.window - sp.shift;
    const int qhi = !a.window || k0 < a.sinks || reach > sp.qlen ? sp.qlen : static_cast<int>(max(reach, int64_t(0)));
    const int t0 = qlo / kBK, t1 = (qhi + kBK - 1) / kBK;
    const int nq = qhi > qlo ? t1 - t0 : 0;
    const int n = nq * a.group;

    Stage<LP, THREADS> qs, ds;
    float lse_r = kInf, delta_r = 0.f;
    const auto load = [&](int it) {
        const int h = kvh * a.group + it / nq, r0 = (t0 + it % nq) * kBK;
        qs.load(a.q + sp.q0 * a.q_row + h * a.q_head, a.q_row, a.d, r0, 0, sp.qlen, 0);
        ds.load(gr.dout + (sp.q0 * a.Hq + h) * static_cast<int64_t>(a.d), static_cast<int64_t>(a.Hq) * a.d, a.d, r0, 0, sp.qlen, 0);
        if (tid < kBK) {
            const int q = r0 + tid;
            lse_r = kInf, delta_r = 0.f;
            if (q < sp.qlen) {
                const int64_t at = (sp.q0 + q) * a.Hq + h;
                const float x = gr.lse[at];
                if (x != -kInf) lse_r = x;
                delta_r = gr.delta[at];
            }
        }
    };
    const auto whole = [&](int r0) {
        const int p = r0 + sp.shift;
        return p - (k0 + KT - 1) >= 0 && (!a.window || p + kBK - 1 - k0 < a.window || k0 + KT <= a.sinks);
    };
    const auto even = [&](int r0) { return whole(r0) && r0 + sp.shift - (k0 + KT - 1) >= a.last; };
    const auto fill = [&](int it) {
        const int buf = it & 1, r0 = (t0 + it % nq) * kBK;
        if (a.buckets && it > 0 && it % nq == 0) {  // another head: its row of the bias
            __syncthreads();
            const int h = kvh * a.group + it / nq;
            for (int i = tid; i < a.buckets; i += THREADS) bias_s[i] = a.bias[static_cast<int64_t>(h) * a.buckets + i];
            __syncthreads();
        }
        qs.store(Qs[buf]);
        ds.store(Ds[buf]);
        if (tid < kBK) {
            lse_s[buf][tid] = lse_r, delta_s[buf][tid] = delta_r;
            const bool any = __any(fabsf(lse_r) > kHuge && fabsf(lse_r) < kInf);
            if (tid == 0) huge_s[buf] = any;
        }
        if (!even(r0)) {
            const int n0 = r0 + sp.shift - (k0 + KT - 1);
            int bucket;
            for (int i = tid; i < TAB - 1; i += THREADS)
                tab[buf][i] = table_entry(a, bounds_s, bias_s, n0 + i, k0 < a.sinks, &bucket);
        }
    };

    f32x16 dk[MB], dv[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) dk[m] = dv[m] = f32x16{};

    for (int i = tid; i < a.buckets; i += THREADS) {
        bounds_s[i] = a.bounds[i];
        bias_s[i] = a.bias[static_cast<int64_t>(kvh) * a.group * a.buckets + i];
    }
    if (n > 0) load(0);
    __syncthreads();
    if (n > 0) fill(0);
    for (int it = 0; it < n; ++it) {
        const int r0 = (t0 + it % nq) * kBK, buf = it & 1;
        if (it + 1 < n) load(it + 1);
        __syncthreads();
        const int p0 = r0 + sp.shift, wkey = k0 + w * 32;  // positions p0 .. p0 + 63, keys wkey .. wkey + 31
        const bool none = p0 + kBK - 1 < wkey || wkey >= sp.klen ||
                          (a.window && p0 - (wkey + 31) >= a.window && wkey >= a.sinks);
        // the last bucket's bias is read before fill() may bring another head's
        const float c = a.buckets ? bias_s[a.buckets - 1] : 0.f;
        if (!none) {
            const bool flat = even(r0), huge = huge_s[buf] != 0;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    Frag q, d;
                    read_row<LP>(q, Qs[buf], 32 * g + ln, 2 * i + half);
                    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q.b, kf[i].b, s, 0, 0, 0);
                    read_row<LP>(d, Ds[buf], 32 * g + ln, 2 * i + half);
                    dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(d.b, vf[i].b, dp, 0, 0, 0);
                }
                // register r: query 32 g + 8 (r / 4) + 4 half + r % 4
                if (flat) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, c);
                } else {
                    const float *tb = tab[buf] + 32 * g + 4 * half + KT - 1 - (w * 32 + ln);
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, tb[8 * (r / 4) + r % 4]);
                    if (wild) {
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (tb[8 * (r / 4) + r % 4] == -kInf) s[r] = -kInf;
                    }
                    if (k0 < a.sinks) {
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int p = p0 + 32 * g + 8 * (r / 4) + 4 * half + r % 4;
                            if (p - kl >= a.window && kl >= a.sinks) s[r] = -kInf;
                        }
                    }
                }
                Frag pf[2], sf[2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const floatx4 l = *reinterpret_cast<const floatx4 *>(&lse_s[buf][32 * g + 8 * j + 4 * half]);
                    const floatx4 e = *reinterpret_cast<const floatx4 *>(&delta_s[buf][32 * g + 8 * j + 4 * half]);
                    float p[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float z = s[4 * j + r];
                        p[r] = huge ? __builtin_amdgcn_exp2f((z - l[r]) * kLog2e)
                                    : __builtin_amdgcn_exp2f(fmaf(z, kLog2e, -l[r] * kLog2e));
                        float x = p[r] * (dp[4 * j + r] - e[r]);
                        if (wild && p[r] == 0.f) x = 0.f;
                        dp[4 * j + r] = x;
                    }
                    pf[j / 2].w[j % 2 * 2] = pack_bf16(p[0], p[1]);
                    pf[j / 2].w[j % 2 * 2 + 1] = pack_bf16(p[2], p[3]);
                    sf[j / 2].w[j % 2 * 2] = pack_bf16(dp[4 * j], dp[4 * j + 1]);
                    sf[j / 2].w[j % 2 * 2 + 1] = pack_bf16(dp[4 * j + 2], dp[4 * j + 3]);
                }
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        Frag x;
                        read_columns<LP>(x, Ds[buf], 32 * g + 16 * u, 32 * m, lane);
                        dv[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.b, pf[u].b, dv[m], 0, 0, 0);
                        read_columns<LP>(x, Qs[buf], 32 * g + 16 * u, 32 * m, lane);
                        dk[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.b, sf[u].b, dk[m], 0, 0, 0);
                    }
            }
        }
        if (it + 1 < n) fill(it + 1);
    }
    if (!live) return;
    const int64_t row = ((sp.k0 + kl) * a.Hkv + kvh) * static_cast<int64_t>(a.d);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * m + 8 * g + 4 * half;
            if (c >= a.d) continue;
            *(DLRM_GLOBAL u32x2 *)(gr.dk + row + c) =
                u32x2{pack_bf16(dk[m][4 * g] * a.scale, dk[m][4 * g + 1] * a.scale),
                      pack_bf16(dk[m][4 * g + 2] * a.scale, dk[m][4 * g + 3] * a.scale)};
            *(DLRM_GLOBAL u32x2 *)(gr.dv + row + c) =
                u32x2{pack_bf16(dv[m][4 * g], dv[m][4 * g + 1]), pack_bf16(dv[m][4 * g + 2], dv[m][4 * g + 3])};
        }
}

// dbias[h][t] = sum over the slots of partial[h][slot][t]: 32 buckets by 32 runs of slots, each in
// order, then the runs in order.
__global__ __launch_bounds__(1024) void k_seq_bias_sum(const float *partial, int64_t slots, int buckets, float *dbias) {
    __shared__ float part[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int t = blockIdx.x * 32 + tx;
    const int64_t h = blockIdx.y;
    float x = 0.f;
    if (t < buckets) {
#pragma unroll 8
        for (int64_t s = ty; s < slots; s += 32) x += partial[(h * slots + s) * buckets + t];
    }
    part[ty][tx] = x;
    __syncthreads();
    if (ty == 0 && t < buckets) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) y += part[i][tx];
        dbias[h * buckets + t] = y;
    }
}

constexpr int kWaves = 4;

size_t delta_bytes(int64_t Nq, int32_t Hq) { return (static_cast<size_t>(Nq) * Hq * 4 + 255) / 256 * 256; }

template <int DP, int LP>
int launch(const Args &a, const Grads &gr, float *dbias, hipStream_t stream) {
    constexpr int NW = kWaves;
    const int64_t qslots = a.B ? slot_count(a.Nq, a.B, NW * 32) : 0, kslots = a.B ? slot_count(a.Nkv, a.B, NW * 32) : 0;
    const int64_t qb = qslots * a.Hq, kb = kslots * a.Hkv;
    if (qb >= (int64_t(1) << 31) - 8 || kb >= (int64_t(1) << 31) - 8) return DLRM_ERR_UNSUPPORTED;
    if (qb > 0) DLRM_LAUNCH("seq_attn_bwd_q", (k_seq_attn_bwd_q<DP, LP, NW>), dim3(round_up_xcd(qb)), dim3(NW * 64), 0, stream, a, gr, qslots);
    if (kb > 0) DLRM_LAUNCH("seq_attn_bwd_kv", (k_seq_attn_bwd_kv<DP, LP, NW>), dim3(round_up_xcd(kb)), dim3(NW * 64), 0, stream, a, gr, kslots);
    if (a.buckets)
        DLRM_LAUNCH("seq_bias_sum", k_seq_bias_sum, dim3((a.buckets + 31) / 32, a.Hq), dim3(1024), 0, stream,
                    static_cast<const float *>(gr.partial), qslots, a.buckets, dbias);
    return launch_status();
}

}  // namespace
}  // namespace seq
}  // namespace dlrm

extern "C" size_t dlrm_seq_attn_bwd_workspace_size(int64_t B, int64_t Nq, int32_t Hq, int32_t buckets) {
    using namespace dlrm::seq;
    if (B < 0 || Nq < 0 || Hq < 1 || buckets < 0 || buckets > DLRM_SEQ_MAX_BUCKETS || B >= (1 << 24) ||
        Nq >= (int64_t(1) << 40) || Hq > 4096)
        return 0;
    const size_t partial = static_cast<size_t>(slot_count(Nq, B, kWaves * 32)) * Hq * buckets * 4;
    return delta_bytes(Nq, Hq) + partial + 256;
}

extern "C" int dlrm_seq_attn_bwd(const dlrm_seq_attn *desc, const uint16_t *dout, const uint16_t *o, const float *o_lo,
                                 const float *lse, uint16_t *dq, uint16_t *dk, uint16_t *dv, float *dbias, void *workspace,
                                 size_t workspace_bytes, dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq;
    Args a;
    const int rc = check_attn(desc, true, &a);
    if (rc != DLRM_OK) return rc;
    if ((a.buckets != 0) != (dbias != nullptr) || !aligned(dbias, 4)) return DLRM_ERR_INVALID_ARG;
    if (a.Nq > 0 && (!dout || !o || !o_lo || !lse || !dq)) return DLRM_ERR_INVALID_ARG;
    if (a.Nkv > 0 && (!dk || !dv)) return DLRM_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(o, 16) || !aligned(o_lo, 16) || !aligned(dq, 16) || !aligned(dk, 16) ||
        !aligned(dv, 16) || !aligned(lse, 4))
        return DLRM_ERR_INVALID_ARG;
    // the keys' tiles are found by the same offsets as the sequences' ends
    const uintptr_t ib = a.idx32 ? 4 : 8;
    if (a.B > 0 && static_cast<const char *>(a.kv_end) != static_cast<const char *>(a.kv_begin) + ib) return DLRM_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < dlrm_seq_attn_bwd_workspace_size(a.B, a.Nq, a.Hq, a.buckets))
        return DLRM_ERR_WORKSPACE;
    Grads gr{};
    gr.dout = dout, gr.o = o, gr.o_lo = o_lo, gr.lse = lse, gr.dq = dq, gr.dk = dk, gr.dv = dv;
    gr.delta = static_cast<float *>(workspace);
    gr.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + delta_bytes(a.Nq, a.Hq));
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    if (a.d <= 32) return launch<32, 32>(a, gr, dbias, stream);
    if (a.d <= 64) return launch<64, 64>(a, gr, dbias, stream);
    return launch<128, 128>(a, gr, dbias, stream);
}
