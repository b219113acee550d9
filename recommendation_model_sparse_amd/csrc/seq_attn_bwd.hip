// Attention over jagged sequences, backward (dlrm_seq.h).
//
//   P = exp(z - lse);  dP = dO V^T;  ds = P (dP - delta), delta = sum_j P dP = <dO, o>
//   dQ = scale ds K;  dK = scale ds^T Q;  dV = P^T dO;  dbias[t] = sum of ds over bucket t
//
// P is computed again from Q, K and the saved log-sums.  Two kernels, so that every sum has an owner
// and no gradient is added to by atomics: one over blocks of queries (delta, dQ, dbias), one over
// blocks of keys (dK, dV; it walks the query heads that share the key head one after the other).
// That computes S and dP twice, with a bias three times (delta, below): 7 products of Q x K x d, or 9,
// instead of the 5 that one kernel with atomic dQ would need.  Both work on the tiles of the forward: the accumulator of S and dP becomes the
// next product's operand in registers, and the transposed operands (K^T; Q^T and dO^T) are read from
// row-major tiles by transposing LDS loads.  As operands P and ds are rounded to bf16, as the matrix
// instruction takes them (fp32's 24 bits would be three products): the gradients are 2.4e-3 from the formulas
// in 64 bits, of which their own rounding to bf16 is 1.7e-3.
//
// delta.  Without a bias it is <dO, o> from the forward's output.  That o is rounded to bf16, which
// the gradients, rounded to bf16 too, bear; dbias does not: it sums ds over up to every pair, where
// most cancels, and would be 1e-3 off (2.2e-7 to 3.6e-7 as it is).  With a bias the first kernel therefore
// goes over its keys twice, first for delta = sum P dP in fp32.  (An output kept in 24 bits by a forward
// that multiplies P in three bf16 pieces was the other way: as much arithmetic, and 6 more bytes an
// element to write and read.)
//
// Bound by waits, as the forward (heads of 64: VALU 25 to 27 %, MFMA 8 %, LDS 13 to 17 %).  Measured,
// for the forward's two cases: over queries 134 and 277 us, of which the sweep for delta takes 36 and 82
// and dbias 38 and 55; over keys 110 and 224, with 27 for the far part of the second.
#include <type_traits>

#include "seq.h"

namespace dlrm {
namespace seq {
namespace {

// Most first keys, and bytes of their sums, that have a far part of their own (below).
constexpr int kFarMost = 128;
constexpr size_t kFarBytes = size_t(256) << 20;

struct Grads {
    const uint16_t *dout, *o;
    const float *lse;
    const int32_t *tiles;  // the sequence of each 64-query tile, from the forward
    float *delta;          // [Nq][Hq]
    float *partial;        // [Hq][slots][buckets]: dbias of each workgroup
    uint16_t *dq, *dk, *dv;
    float *split;          // [splits][2][Nkv][Hkv][d]: dk and dv, where a key block's queries are split
    int splits;
    // first keys under a window: their gradients from the queries past it, [slot][Hkv][far_sinks][2][d]
    float *far;
    int far_sinks;
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

// WQ wavefronts of 32 queries, by WK that take one half each of a tile's 64 keys.
template <int DP, int LP, int WQ, int WK, int OCC, int NEAR>
__global__ __launch_bounds__(WQ * WK * 64, OCC) void k_seq_attn_bwd_q(const Args a, const Grads gr) {
    constexpr int QT = WQ * 32, STEPS = DP / 16, MB = DP / 32, THREADS = WQ * WK * 64, NW = WQ * WK;
    constexpr int TAB = QT + kBK, TILE = kBK * kPitch<LP>, PITCH = 36;
    static_assert(QT == kQT, "the forward's tiles");
    __shared__ __attribute__((aligned(16))) uint16_t tiles_s[2 * TILE];
    __shared__ __attribute__((aligned(16))) float skew[NW][16 * PITCH];
    __shared__ float near_s[kPad + NEAR], tab[TAB], sums[NW][DLRM_SEQ_MAX_BUCKETS], half_s[WK == 2 ? WQ : 1][32];
    __shared__ uint8_t bnear_s[kPad + NEAR], btab[TAB];
    uint16_t *const Ks = tiles_s, *const Vs = tiles_s + TILE;
    int *const bounds_s = reinterpret_cast<int *>(tiles_s);  // before the first tile
    float *const bias_s = reinterpret_cast<float *>(tiles_s) + DLRM_SEQ_MAX_BUCKETS;

    const int slots = static_cast<int>(slot_count(a.Nq, a.B, QT));
    const int slot = static_cast<int>(xcd_contiguous(blockIdx.x, gridDim.x));
    if (slot >= slots) return;
    const int h = blockIdx.y;
    const int64_t id = static_cast<int64_t>(h) * slots + slot;
    const int b = min(max(gr.tiles[slot], 0), a.B - 1);
    const Span sp = span_of(a, b);
    const int t = slot - (static_cast<int>(sp.q0) / QT + b);
    const int tiles = (sp.qlen + QT - 1) / QT;
    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, half = lane >> 5;
    if (t < 0 || t >= tiles) {
        for (int i = tid; i < a.buckets; i += THREADS) gr.partial[id * a.buckets + i] = 0.f;
        return;
    }
    const int q0 = (tiles - 1 - t) * QT;
    const int wave = static_cast<int>(wave_id()), w = wave % WQ, wk = wave / WQ;
    const int kvh = h / a.group;
    const uint16_t *kb = a.k + sp.k0 * a.k_row + kvh * a.k_head;
    const uint16_t *vb = a.v + sp.k0 * a.v_row + kvh * a.v_head;

    const int pmin = q0 + sp.shift, pmax = min(q0 + QT, sp.qlen) - 1 + sp.shift;
    const int end = min(sp.klen, pmax + 1);
    const int first = a.window ? max(0, pmin - a.window + 1) : 0;
    const int t1 = end > 0 ? (end + kBK - 1) / kBK : 0;
    const int t0 = min(first / kBK, t1);
    const int nsink = min((a.sinks + kBK - 1) / kBK, t0);
    const int n = nsink + t1 - t0;

    Stage<LP, THREADS> ks(a.k_row, a.d), vs(a.v_row, a.d);
    const auto key0 = [&](int it) { return (it < nsink ? it : t0 + it - nsink) * kBK; };
    const auto load = [&](int it) {
        ks.load(kb, a.k_row, a.d, key0(it), first, end, a.sinks);
        vs.load(vb, a.v_row, a.d, key0(it), first, end, a.sinks);
    };
    const auto even = [&](int k0) {
        const int nearest = pmin - (k0 + kBK - 1);
        return nearest >= a.last && (!a.window || q0 + QT - 1 + sp.shift - k0 < a.window || k0 + kBK <= a.sinks);
    };
    const auto close = [&](int k0) { return pmin - k0 + QT - 1 < NEAR && k0 >= a.sinks; };
    const float *const bias_row = a.buckets ? a.bias + static_cast<int64_t>(h) * a.buckets : nullptr;
    const float last_bias = a.buckets ? bias_row[a.buckets - 1] : 0.f;
    const auto table = [&](int k0) {
        if (even(k0) || close(k0)) return;
        const int n0 = pmin - (k0 + kBK - 1);
        for (int i = tid; i < TAB - 1; i += THREADS) {
            int bucket;
            tab[i] = bias_at(a, a.bounds, bias_row, n0 + i, k0 < a.sinks, &bucket);
            btab[i] = static_cast<uint8_t>(bucket);
        }
    };

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
            if (!a.buckets) {
                const u32x4 x = *(const DLRM_GLOBAL u32x4 *)(gr.o + orow + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    delta = fmaf(bf16_lo(df[s].w[e]), bf16_lo(x[e]), delta);
                    delta = fmaf(bf16_hi(df[s].w[e]), bf16_hi(x[e]), delta);
                }
            }
        }
    }
    if (live) {
        const float x = gr.lse[(sp.q0 + ql) * a.Hq + h];
        if (x != -kInf) lse = x;
    }
    delta = add_halves(delta);
    const bool huge = __any(fabsf(lse) > kHuge && fabsf(lse) < kInf);
    const float lse2 = lse * kLog2e;
    for (int i = tid; i < a.buckets; i += THREADS) {
        bounds_s[i] = a.bounds[i];
        bias_s[i] = bias_row[i];
    }
    __syncthreads();
    {
        const int reach = n > 0 ? min(NEAR, pmin + QT - t0 * kBK) : 0;
        for (int i = tid; i < reach; i += THREADS) {
            int bucket;
            near_s[kPad + i] = bias_at(a, bounds_s, bias_s, i, false, &bucket);
            bnear_s[kPad + i] = static_cast<uint8_t>(bucket);
        }
        for (int i = tid; i < kPad; i += THREADS) near_s[i] = -kInf, bnear_s[i] = 0;
    }

    f32x16 dq[MB];
    float far = 0.f;  // ds summed over the pairs of the last bucket, where a tile has only those
    const uint16_t *const krow = Ks + row_base<LP>(ln, half), *const vrow = Vs + row_base<LP>(ln, half);
    const uint16_t *const kcol = Ks + column_base<LP>(lane);

    // One pass over the keys: for delta alone, or for the gradients.  WILD as in the forward.
    const auto sweep = [&](auto is_wild, auto is_delta, bool staged) {
        constexpr bool WILD = decltype(is_wild)::value, DELTA = decltype(is_delta)::value;
        for (int it = 0; it < n; ++it) {
            const int k0 = key0(it);
            if (!staged) {
                load(it);
                __syncthreads();
                table(k0);
                ks.store(Ks);
                vs.store(Vs);
                __syncthreads();
            }
            const bool by_near = close(k0);
            const int wpos = pmin + w * 32;
            const bool flat = even(k0);
#pragma unroll 1
            for (int g = WK == 2 ? wk : 0; g < (WK == 2 ? wk + 1 : 2); ++g) {
                const int k1 = k0 + 32 * g;
                if (wpos + 31 < k1 || q0 + w * 32 >= sp.qlen || (a.window && wpos - (k1 + 31) >= a.window && k1 >= a.sinks))
                    continue;
                const int at = 32 * g * kPitch<LP>;
                f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    Frag k, v;
                    read_row(k, krow + at, i);
                    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k.b, qf[i].b, s, 0, 0, 0);
                    read_row(v, vrow + at, i);
                    dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, df[i].b, dp, 0, 0, 0);
                }
                if (flat) {
                    #pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, last_bias);
                } else {
                    const float *tb = by_near ? near_s + kPad + wpos - k1 + ln - 4 * half
                                              : tab + w * 32 + ln + kBK - 1 - 32 * g - 4 * half;
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
                            const int key = k1 + 8 * (r / 4) + 4 * half + r % 4;
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
                if constexpr (WILD) {  // a hidden key's dP may be NaN
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (s[r] == 0.f) dp[r] = delta;
                }
                if constexpr (DELTA) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) far = fmaf(s[r], dp[r], far);
                    continue;
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) dp[r] = s[r] * (dp[r] - delta);
                Frag ds[2];
#pragma unroll
                for (int r = 0; r < 16; r += 2) ds[r / 8].w[r / 2 % 4] = pack_bf16(dp[r], dp[r + 1]);
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        Frag k;
                        read_columns<LP>(k, kcol + at, 16 * u, 32 * m);
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
                    // distance D + ln, the others at D + ln - 32, D = wpos - k1.
                    float *sk = skew[wave];
                    float upper = 0.f, lower = 0.f;
#pragma unroll
                    for (int q16 = 0; q16 < 32; q16 += 16) {  // 16 queries at a time, for LDS's sake
                        wave_lds_sync();
                        if ((ln & 16) == q16) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<floatx4 *>(sk + (ln & 15) * PITCH + 8 * j + 4 * half) =
                                    floatx4{dp[4 * j], dp[4 * j + 1], dp[4 * j + 2], dp[4 * j + 3]};
                        }
                        wave_lds_sync();
                        const int edge = ln - q16 - 8 * half;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float x = sk[(8 * half + i) * PITCH + ((q16 + 8 * half + i - ln) & 31)];
                            upper += i >= edge ? x : 0.f;
                            lower += i >= edge ? 0.f : x;
                        }
                    }
                    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(lower), __float_as_uint(upper), false, false);
                    const float x = __uint_as_float(r[0]) + __uint_as_float(r[1]);  // distance D - 32 + lane
                    // (no pair is at distance D - 32: lane 0 adds a zero, and may stay inside the tile's table)
                    add_by_bucket(sums[wave], x,
                                  by_near ? bnear_s[kPad + wpos - k1 - 32 + lane] : btab[max(w * 32 + 31 - 32 * g + lane, 0)], lane);
                }
            }
        }
    };
    const auto both = [&](auto is_wild, bool staged) {
        if (a.buckets) {
            far = delta = 0.f;
            sweep(is_wild, std::true_type(), staged);
            staged = n == 1;  // its only tile is still there
            delta = add_halves(far);
            if constexpr (WK == 2) {
                __syncthreads();
                if (wk == 1 && half == 0) half_s[w][ln] = delta;
                __syncthreads();
                const float x = half_s[w][ln];
                if (wk == 0) delta += x;
                __syncthreads();
                if (wk == 0 && half == 0) half_s[w][ln] = delta;
                __syncthreads();
                delta = half_s[w][ln];
            }
        }
        far = 0.f;
#pragma unroll
        for (int m = 0; m < MB; ++m) dq[m] = f32x16{};
        for (int i = lane; i < a.buckets; i += 64) sums[wave][i] = 0.f;
        wave_lds_sync();
        sweep(is_wild, std::false_type(), staged);
    };
    both(std::false_type(), false);
    float any = 0.f;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) any += dq[m][r];
    if (__syncthreads_or(any != any)) {
            both(std::true_type(), false);
    }
    if (a.buckets) {
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) far += __shfl_xor(far, i);
        if (lane == 0) sums[wave][a.buckets - 1] += far;
    }
    __syncthreads();
    for (int i = tid; i < a.buckets; i += THREADS) {
        float x = 0.f;
#pragma unroll
        for (int v = 0; v < NW; ++v) x += sums[v][i];
        gr.partial[id * a.buckets + i] = x;
    }
    if constexpr (WK == 2) {
        float *const part = reinterpret_cast<float *>(tiles_s) + w * MB * 16 * 64 + lane;
        static_assert(WQ * MB * 16 * 64 * 4 <= 2 * TILE * 2, "the tiles' room holds the halves' results");
        if (wk == 1) {
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int r = 0; r < 16; ++r) part[(m * 16 + r) * 64] = dq[m][r];
        }
        __syncthreads();
        if (wk == 1) return;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) dq[m][r] += part[(m * 16 + r) * 64];
    }
    if (!live) return;
    if (half == 0) gr.delta[(sp.q0 + ql) * a.Hq + h] = delta;
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

// WY wavefronts of 32 keys, by WX that take one half each of a tile's 64 queries.  blockIdx.y: the
// key head, and which run of the queries (of all heads that share it) where they are split.
//
// OWN: the block's values are read from LDS at every step instead of kept in registers: at heads of 128
// 47 fewer registers spill, which leaves 22 (252 -> 224 us on 4 sequences of 2000 to 4096, 8 heads over 2;
// the keys in LDS too: 228), at heads of 64 a third wavefront fits a SIMD, with 12 (114 -> 110 us on 1024
// sequences of 16 to 512, 2 heads).  Heads of 32 fit as they are.
//
// FAR: the few first keys that every later query sees, and only the queries past the window: a key
// block of its own would walk all queries of a long sequence after the others are done (4 sequences of
// up to 4096 under a window of 1024: 1367 us with that, 35 + 252 us as it is).  A workgroup takes one of
// the forward's tiles of queries; the block that owns the keys adds their sums in order.
template <int DP, int LP, int WY, int WX, int OCC, bool OWN, bool FAR>
__global__ __launch_bounds__(WY * WX * 64, OCC) void k_seq_attn_bwd_kv(const Args a, const Grads gr) {
    constexpr int KT = WY * 32, STEPS = DP / 16, MB = DP / 32, THREADS = WY * WX * 64;
    constexpr int TAB = KT + kBK, TILE = kBK * kPitch<LP>;
    __shared__ __attribute__((aligned(16))) uint16_t tiles_s[2 * TILE];
    __shared__ __attribute__((aligned(16))) float lse_s[kBK], delta_s[kBK];
    __shared__ float tab[2][TAB], bias_s[2][DLRM_SEQ_MAX_BUCKETS];
    __shared__ int bounds_s[DLRM_SEQ_MAX_BUCKETS];
    __shared__ __attribute__((aligned(16))) uint16_t own_s[OWN ? KT * kPitch<LP> : 8];
    uint16_t *const Qs = tiles_s, *const Ds = tiles_s + TILE;

    const int slot = static_cast<int>(xcd_contiguous(blockIdx.x, gridDim.x));
    if (FAR && slot >= slot_count(a.Nq, a.B, kQT)) return;
    const int b = FAR ? min(max(gr.tiles[slot], 0), a.B - 1) : find_sequence(a, a.kv_begin, a.Nkv, slot, KT);
    const Span sp = span_of(a, b);
    int kvh, run = 0, k0, qlo, qhi;
    if constexpr (FAR) {
        const int blocks = (gr.far_sinks + KT - 1) / KT, c = slot - (static_cast<int>(sp.q0) / kQT + b);
        kvh = blockIdx.y / blocks, k0 = blockIdx.y % blocks * KT;
        qlo = max(c * kQT, k0 + a.window - sp.shift);
        qhi = min((c + 1) * kQT, sp.qlen);
        if (c < 0 || k0 >= sp.klen || qlo >= qhi) return;
    } else {
        kvh = blockIdx.y / gr.splits, run = blockIdx.y % gr.splits;
        const int t = slot - (static_cast<int>(sp.k0) / KT + b);
        if (t < 0 || t * KT >= sp.klen) return;
        k0 = t * KT;  // the first keys are seen by the most queries: first
        qlo = max(0, k0 - sp.shift);
        const int64_t reach = static_cast<int64_t>(k0) + KT - 1 + a.window - sp.shift;
        qhi = !a.window || k0 < a.sinks || reach > sp.qlen ? sp.qlen : static_cast<int>(max(reach, int64_t(0)));
    }

    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, half = lane >> 5;
    const int wave = static_cast<int>(wave_id()), w = wave % WY, wx = wave / WY;
    const int kl = k0 + w * 32 + ln;
    const bool live = kl < sp.klen;
    const int t0 = qlo / kBK, nq = qhi > qlo ? (qhi + kBK - 1) / kBK - t0 : 0;
    // the tiles of every head in a row, and this workgroup's run of them
    const int all = nq * a.group;
    const int i0 = static_cast<int>(static_cast<int64_t>(all) * run / (FAR ? 1 : gr.splits));
    const int i1 = static_cast<int>(static_cast<int64_t>(all) * (run + 1) / (FAR ? 1 : gr.splits));

    Stage<LP, THREADS> qs(a.q_row, a.d), ds(static_cast<int64_t>(a.Hq) * a.d, a.d);
    float lse_r = kInf, delta_r = 0.f;
    const auto load = [&](int it) {
        const int h = kvh * a.group + it / nq, r0 = (t0 + it % nq) * kBK;
        qs.load(a.q + sp.q0 * a.q_row + h * a.q_head, a.q_row, a.d, r0, 0, sp.qlen, 0);
        ds.load(gr.dout + (sp.q0 * a.Hq + h) * static_cast<int64_t>(a.d), static_cast<int64_t>(a.Hq) * a.d, a.d, r0, 0, sp.qlen, 0);
        if (tid < kBK) {
            const int q = r0 + tid;
            lse_r = kInf, delta_r = 0.f;
            if (q < sp.qlen && (!FAR || (q >= qlo && q < qhi))) {
                const int64_t at = (sp.q0 + q) * a.Hq + h;
                const float x = gr.lse[at];
                if (x != -kInf) lse_r = x;
                delta_r = gr.delta[at];
            }
        }
    };
    const auto row_of_bias = [&](int it) {
        const int h = it / nq;
        for (int i = tid; i < a.buckets; i += THREADS)
            bias_s[h & 1][i] = a.bias[static_cast<int64_t>(kvh * a.group + h) * a.buckets + i];
    };
    const auto even = [&](int r0) {
        const int nearest = r0 + sp.shift - (k0 + KT - 1);
        if (FAR) return nearest >= a.last && nearest >= a.window && k0 + KT <= a.sinks;
        return nearest >= a.last && (!a.window || r0 + sp.shift + kBK - 1 - k0 < a.window || k0 + KT <= a.sinks);
    };
    const auto table = [&](int it) {
        const int r0 = (t0 + it % nq) * kBK, n0 = r0 + sp.shift - (k0 + KT - 1);
        if (even(r0)) return;
        for (int i = tid; i < TAB - 1; i += THREADS) {
            int bucket;
            float x = bias_at(a, bounds_s, bias_s[it / nq & 1], n0 + i, k0 < a.sinks, &bucket);
            if (FAR && n0 + i < a.window) x = -kInf;
            tab[it & 1][i] = x;
        }
    };

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
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            odd |= only_finite(kf[s].w[e]) != kf[s].w[e] || only_finite(vf[s].w[e]) != vf[s].w[e];
    // An infinity or NaN in a key makes its gradients NaN, from hidden queries too (0 * NaN): right where
    // a query sees it; where none does, the zeros are put in at the end.
    const auto unseen = [&] {
        const bool any = (__ballot(odd) >> ln & 0x100000001ull) != 0;
        const int least = max(0, sp.shift - kl);  // distance to the first query that is not before the key
        return any && (sp.qlen == 0 || (a.window && least >= a.window && kl >= max(a.sinks, gr.far_sinks)));
    };

    const uint16_t *const own_row = own_s + w * 32 * kPitch<LP> + row_base<LP>(ln, half);
    if constexpr (OWN) {  // the barrier before the first table orders it
        uint16_t *const to = own_s + w * 32 * kPitch<LP> + row_base<LP>(ln, half);
        if (wx == 0) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) *reinterpret_cast<u32x4 *>(to + 16 * s) = vf[s].q;
        }
    }

    f32x16 dk[MB], dv[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) dk[m] = dv[m] = f32x16{};
    const int rows = row_base<LP>(ln, half), cols = column_base<LP>(lane);
    const float *const tb0 = tab[0] + 4 * half + KT - 1 - (w * 32 + ln);

    for (int i = tid; i < a.buckets; i += THREADS) bounds_s[i] = a.bounds[i];
    if (i1 > i0) row_of_bias(i0);
    __syncthreads();
    if (i1 > i0) table(i0);
    for (int it = i0; it < i1; ++it) {
        const int r0 = (t0 + it % nq) * kBK;
        if (it > i0) __syncthreads();  // the tile before has been read
        load(it);
        qs.store(Qs);
        ds.store(Ds);
        if (tid < kBK) lse_s[tid] = lse_r, delta_s[tid] = delta_r;
        if (it + 1 < i1 && (it + 1) % nq == 0) row_of_bias(it + 1);
        __syncthreads();
        if (it + 1 < i1) {
            table(it + 1);
        }
        const bool flat = even(r0);
        const int wkey = k0 + w * 32;
        const float c = a.buckets ? bias_s[it / nq & 1][a.buckets - 1] : 0.f;
#pragma unroll 1
        for (int g = WX == 2 ? wx : 0; g < (WX == 2 ? wx + 1 : 2); ++g) {
            const int p0 = r0 + 32 * g + sp.shift;  // positions p0 .. p0 + 31, keys wkey .. wkey + 31
            if (p0 + 31 < wkey || wkey >= sp.klen || r0 + 32 * g >= qhi) continue;
            if (FAR ? wkey >= a.sinks || p0 + 31 - wkey < a.window : a.window && p0 - (wkey + 31) >= a.window && wkey >= a.sinks)
                continue;
            const uint16_t *const qt = Qs + 32 * g * kPitch<LP>, *const dt = Ds + 32 * g * kPitch<LP>;
            f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                Frag q, d, v = vf[i];
                if constexpr (OWN) read_row(v, own_row, i);
                read_row(q, qt + rows, i);
                s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q.b, kf[i].b, s, 0, 0, 0);
                read_row(d, dt + rows, i);
                dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(d.b, v.b, dp, 0, 0, 0);
            }
            // register r: query 8 (r / 4) + 4 half + r % 4
            if (flat) {
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, c);
            } else {
                const float *tb = tb0 + (it & 1) * TAB + 32 * g;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, tb[8 * (r / 4) + r % 4]);
                if (k0 < a.sinks) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int p = p0 + 8 * (r / 4) + 4 * half + r % 4;
                        if (p - kl >= a.window && kl >= a.sinks) s[r] = -kInf;
                    }
                }
            }
            Frag pf[2], sf[2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const floatx4 l = *reinterpret_cast<const floatx4 *>(&lse_s[32 * g + 8 * j + 4 * half]);
                const floatx4 e = *reinterpret_cast<const floatx4 *>(&delta_s[32 * g + 8 * j + 4 * half]);
                float p[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    p[r] = __builtin_amdgcn_exp2f((s[4 * j + r] - l[r]) * kLog2e);
                    dp[4 * j + r] = p[r] * (dp[4 * j + r] - e[r]);
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
                    read_columns<LP>(x, dt + cols, 16 * u, 32 * m);
                    dv[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.b, pf[u].b, dv[m], 0, 0, 0);
                    read_columns<LP>(x, qt + cols, 16 * u, 32 * m);
                    dk[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.b, sf[u].b, dk[m], 0, 0, 0);
                }
        }
    }
    if constexpr (WX == 2) {  // the second half of the queries joins the first, dk and then dv
        float *const part = reinterpret_cast<float *>(tiles_s) + w * MB * 16 * 64 + lane;
        static_assert(WY * MB * 16 * 64 * 4 <= 2 * TILE * 2, "the tiles' room holds the halves' results");
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            f32x16 *const g = x ? dv : dk;
            __syncthreads();
            if (wx == 1) {
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int r = 0; r < 16; ++r) part[(m * 16 + r) * 64] = g[m][r];
            }
            __syncthreads();
            if (wx == 0) {
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int r = 0; r < 16; ++r) g[m][r] += part[(m * 16 + r) * 64];
            }
        }
        if (wx == 1) return;
    }
    if (!live) return;
    if constexpr (FAR) {
        if (kl >= a.sinks) return;
        float *const out = gr.far + ((static_cast<int64_t>(slot) * a.Hkv + kvh) * gr.far_sinks + kl) * 2 * a.d;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = 32 * m + 8 * g + 4 * half;
                if (c >= a.d) continue;
                *(DLRM_GLOBAL floatx4 *)(out + c) = floatx4{dk[m][4 * g], dk[m][4 * g + 1], dk[m][4 * g + 2], dk[m][4 * g + 3]};
                *(DLRM_GLOBAL floatx4 *)(out + a.d + c) = floatx4{dv[m][4 * g], dv[m][4 * g + 1], dv[m][4 * g + 2], dv[m][4 * g + 3]};
            }
        return;
    }
    if (kl < gr.far_sinks && run == 0) {
        const int past = max(0, k0 + a.window - sp.shift), base = static_cast<int>(sp.q0) / kQT + b;
        for (int c = past / kQT; past < sp.qlen && c * kQT < sp.qlen; ++c) {
            const float *in = gr.far + ((static_cast<int64_t>(base + c) * a.Hkv + kvh) * gr.far_sinks + kl) * 2 * a.d;
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int col = 32 * m + 8 * g + 4 * half;
                    if (col >= a.d) continue;
                    const floatx4 x = *(const DLRM_GLOBAL floatx4 *)(in + col), y = *(const DLRM_GLOBAL floatx4 *)(in + a.d + col);
#pragma unroll
                    for (int r = 0; r < 4; ++r) dk[m][4 * g + r] += x[r], dv[m][4 * g + r] += y[r];
                }
        }
    }
    const int64_t row = ((sp.k0 + kl) * a.Hkv + kvh) * static_cast<int64_t>(a.d), plane = a.Nkv * a.Hkv * a.d;
    const bool clear = unseen();
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * m + 8 * g + 4 * half;
            if (c >= a.d) continue;
            floatx4 x, y;
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = clear ? 0.f : dk[m][4 * g + r] * a.scale, y[r] = clear ? 0.f : dv[m][4 * g + r];
            if (gr.splits > 1) {
                *(DLRM_GLOBAL floatx4 *)(gr.split + 2 * run * plane + row + c) = x;
                *(DLRM_GLOBAL floatx4 *)(gr.split + (2 * run + 1) * plane + row + c) = y;
            } else {
                *(DLRM_GLOBAL u32x2 *)(gr.dk + row + c) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
                *(DLRM_GLOBAL u32x2 *)(gr.dv + row + c) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
            }
        }
}

// dk, dv = the sums over the runs, in order; four elements a thread of each.  Only the sequences' rows:
// the runs wrote no others, and the caller's are not to be touched.
__global__ __launch_bounds__(256) void k_seq_kv_sum(const Args a, const float *split, int splits, int64_t plane, uint16_t *dk, uint16_t *dv) {
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4, width = static_cast<int64_t>(a.Hkv) * a.d;
    if (e < offset_at(a, a.kv_begin, 0, a.Nkv) * width || e >= offset_at(a, a.kv_begin, a.B, a.Nkv) * width) return;
    floatx4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
    for (int s = 0; s < splits; ++s) {
        x += *(const DLRM_GLOBAL floatx4 *)(split + 2 * s * plane + e);
        y += *(const DLRM_GLOBAL floatx4 *)(split + (2 * s + 1) * plane + e);
    }
    *(DLRM_GLOBAL u32x2 *)(dk + e) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    *(DLRM_GLOBAL u32x2 *)(dv + e) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
}

// dbias[h][t] = sum over the slots of partial[h][slot][t]: 8 buckets by 128 runs of slots, each in
// order, then the runs in order.
__global__ __launch_bounds__(1024) void k_seq_bias_sum(const float *partial, int64_t slots, int buckets, float *dbias) {
    __shared__ float part[128][9];
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
    const int t = blockIdx.x * 8 + tx;
    const int64_t h = blockIdx.y;
    float x = 0.f;
    if (t < buckets) {
#pragma unroll 8
        for (int64_t s = ty; s < slots; s += 128) x += partial[(h * slots + s) * buckets + t];
    }
    part[ty][tx] = x;
    __syncthreads();
    if (ty < 8) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) y += part[16 * ty + i][tx];
        part[16 * ty][tx] = y;
    }
    __syncthreads();
    if (ty == 0 && t < buckets) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y += part[16 * i][tx];
        dbias[h * buckets + t] = y;
    }
}

// The workspace: delta, the partial dbias, the split and the far sums of dk and dv.
struct Layout {
    int64_t qslots, kslots;
    int splits, far_sinks;
    size_t partial, split, far, bytes;
};

constexpr int kKT = 64;  // keys of a workgroup

Layout layout_of(const Args &a) {
    Layout l{};
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    // no queries: the forward wrote no tiles, and nothing may look a slot up in them
    l.qslots = a.B && a.Nq ? slot_count(a.Nq, a.B, kQT) : 0, l.kslots = a.B && a.Nkv ? slot_count(a.Nkv, a.B, kKT) : 0;
    // a key block's queries are split where there are fewer blocks than two a CU, down to four tiles each
    // (4 sequences of 2000 to 4096, 8 heads of 128 over 2: unsplit 331 us, in 2 runs 254 and 11 for the
    // sum, in 4 263 and 18, in 8 291 and 31)
    const int64_t blocks = l.kslots * a.Hkv, tiles = l.kslots ? a.group * (a.Nq / a.B / kBK) : 0;
    l.splits = 1;
    while (l.splits < 8 && blocks * l.splits < 512 && tiles >= 8 * l.splits) l.splits *= 2;
    size_t far = a.sinks <= kFarMost ? static_cast<size_t>(l.qslots) * a.Hkv * a.sinks * 2 * a.d * 4 : 0;
    if (far > kFarBytes) far = 0;
    l.far_sinks = far ? a.sinks : 0;
    l.partial = up(static_cast<size_t>(a.Nq) * a.Hq * 4);
    l.split = l.partial + up(static_cast<size_t>(l.qslots) * a.Hq * a.buckets * 4);
    l.far = l.split + (l.splits > 1 ? up(static_cast<size_t>(l.splits) * 2 * a.Nkv * a.Hkv * a.d * 4) : 0);
    l.bytes = l.far + up(far) + 256;
    return l;
}

template <int DP, int LP, int WK, int WX, int O1, int O2, bool OWN, int NEAR>
int launch(const Args &a, const Grads &g, const Layout &l, float *dbias, hipStream_t stream) {
    if (l.qslots > 0)
        DLRM_LAUNCH("seq_attn_bwd_q", (k_seq_attn_bwd_q<DP, LP, 2, WK, O1, NEAR>), dim3(round_up_xcd(l.qslots), a.Hq), dim3(128 * WK), 0,
                    stream, a, g);
    Args near = a;
    if (l.far_sinks && l.qslots > 0) {
        DLRM_LAUNCH("seq_attn_bwd_far", (k_seq_attn_bwd_kv<DP, LP, 2, WX, O2, OWN, true>),
                    dim3(round_up_xcd(l.qslots), a.Hkv * ((l.far_sinks + kKT - 1) / kKT)), dim3(128 * WX), 0, stream, a, g);
        near.sinks = 0;  // what is left of the first keys' queries is the window's
    }
    if (l.kslots > 0)
        DLRM_LAUNCH("seq_attn_bwd_kv", (k_seq_attn_bwd_kv<DP, LP, 2, WX, O2, OWN, false>), dim3(round_up_xcd(l.kslots), a.Hkv * l.splits),
                    dim3(128 * WX), 0, stream, near, g);
    const int64_t plane = a.Nkv * a.Hkv * a.d;
    if (l.splits > 1)
        DLRM_LAUNCH("seq_kv_sum", k_seq_kv_sum, dim3(static_cast<uint32_t>((plane / 4 + 255) / 256)), dim3(256), 0, stream,
                    a, static_cast<const float *>(g.split), l.splits, plane, g.dk, g.dv);
    if (a.buckets)
        DLRM_LAUNCH("seq_bias_sum", k_seq_bias_sum, dim3((a.buckets + 7) / 8, a.Hq), dim3(1024), 0, stream,
                    static_cast<const float *>(g.partial), l.qslots, a.buckets, dbias);
    return launch_status();
}

}  // namespace
}  // namespace seq
}  // namespace dlrm

extern "C" size_t dlrm_seq_attn_bwd_workspace_size(const dlrm_seq_attn *desc) {
    using namespace dlrm::seq;
    Args a;
    return check_attn(desc, true, &a) == DLRM_OK ? layout_of(a).bytes : 0;
}

extern "C" int dlrm_seq_attn_bwd(const dlrm_seq_attn *desc, const uint16_t *dout, const uint16_t *o, const float *lse,
                                 const int32_t *tiles, uint16_t *dq, uint16_t *dk, uint16_t *dv, float *dbias, void *workspace,
                                 size_t workspace_bytes, dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq;
    Args a;
    const int rc = check_attn(desc, true, &a);
    if (rc != DLRM_OK) return rc;
    if ((a.buckets != 0) != (dbias != nullptr) || !aligned(dbias, 4)) return DLRM_ERR_INVALID_ARG;
    if (a.Nq > 0 && (!dout || !o || !lse || !dq || (a.B > 0 && !tiles))) return DLRM_ERR_INVALID_ARG;
    if (a.Nkv > 0 && (!dk || !dv)) return DLRM_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(o, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(lse, 4) ||
        !aligned(tiles, 4))
        return DLRM_ERR_INVALID_ARG;
    // the keys' tiles are found by the same offsets as the sequences' ends
    const uintptr_t ib = a.idx32 ? 4 : 8;
    if (a.B > 0 && static_cast<const char *>(a.kv_end) != static_cast<const char *>(a.kv_begin) + ib) return DLRM_ERR_INVALID_ARG;
    const Layout l = layout_of(a);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < l.bytes) return DLRM_ERR_WORKSPACE;
    if (l.qslots == 0 && l.kslots == 0 && !a.buckets) return DLRM_OK;
    char *const ws = static_cast<char *>(workspace);
    Grads g{};
    g.dout = dout, g.o = o, g.lse = lse, g.tiles = tiles, g.dq = dq, g.dk = dk, g.dv = dv;
    g.delta = reinterpret_cast<float *>(ws), g.partial = reinterpret_cast<float *>(ws + l.partial);
    g.split = reinterpret_cast<float *>(ws + l.split), g.splits = l.splits;
    g.far = reinterpret_cast<float *>(ws + l.far), g.far_sinks = l.far_sinks;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    // Wavefronts that share a tile: two more at heads of 128 (over queries 361 us against 437 with 2; over
    // keys 336 either way), none at 64 (149 against 191, and 119 against 173).  The near biases: 2048
    // distances for 896 at heads of 32, 197 -> 178 us, for 1280 at 128, 240 -> 229, for 384 at 64, 240 ->
    // 204 (8 sequences of 2048, 4 heads, a bias that differs up to 2048), but there they cost a workgroup a
    // CU: 134 -> 146 (1024 sequences of 16 to 512) where 384 reach past all that is not even.
    if (a.d <= 32) return launch<32, 32, 1, 1, 3, 2, false, 2048>(a, g, l, dbias, stream);
    const int uneven = a.window && a.window < a.last ? a.window : a.last;  // distances of differing biases, or hidden ones
    if (a.d <= 64 && uneven + 2 * kBK <= 384) return launch<64, 64, 1, 1, 3, 3, true, 384>(a, g, l, dbias, stream);
    if (a.d <= 64) return launch<64, 64, 1, 1, 2, 3, true, 2048>(a, g, l, dbias, stream);
    return launch<128, 128, 2, 2, 2, 2, true, 2048>(a, g, l, dbias, stream);
}
