// Attention over jagged sequences, forward (dlrm_seq.h), and the checks that the attention calls
// share.
//
//   z = scale <q, k> + bias(distance);  P = exp(z - max);  o = sum P v / sum P
//
// One pass over the keys with a running maximum and sum.  A wavefront owns 32 queries and works on
// transposed tiles: S^T = K Q^T has one query a lane (32x32x16 matrix instructions, the
// accumulator's column), so the maximum and the sum of a row are sums over registers and one
// exchange between lanes l and l + 32, and P^T is, as it stands in the registers, the second
// operand of O^T = V^T P^T.  P never goes through LDS; V^T is read from the row-major tile of V by
// transposing LDS loads.  P is rounded to bf16 there, as the matrix instruction takes it (fp32's 24 bits would
// be three products): o is 2.0e-3 from the formula in 64 bits, of which its own rounding to bf16 is 1.6e-3.
//
// Bound by waits, half of the wavefronts' cycles: no unit is busy for a third of the time (heads of 64:
// VALU 30 %, MFMA 7 %, LDS 13 %; of 128: 22, 12, 23).  Measured: 1024 sequences of 16 to 512, 2 heads of
// 64, 64 us (145 TFLOP/s of the visible pairs' products); 4 of 2000 to 4096, window 1024, 8 heads of 128
// over 2, 121 us (302).
#include <type_traits>

#include "seq.h"

namespace dlrm {
namespace seq {

int check_attn(const dlrm_seq_attn *a, bool need_q_offsets, Args *out) {
    if (!a) return DLRM_ERR_INVALID_ARG;
    if (a->B < 0 || a->Nq < 0 || a->Nkv < 0 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv != 0 || a->d < 1)
        return DLRM_ERR_INVALID_ARG;
    if (a->index_type != DLRM_INDEX_I64 && a->index_type != DLRM_INDEX_I32) return DLRM_ERR_INVALID_ARG;
    if (a->window < 0 || a->sinks < 0 || !(a->scale == a->scale)) return DLRM_ERR_INVALID_ARG;
    if (a->bias) {
        if (!a->bounds || a->buckets < 1 || a->bounds[0] != 0) return DLRM_ERR_INVALID_ARG;
        if (a->buckets > DLRM_SEQ_MAX_BUCKETS) return DLRM_ERR_UNSUPPORTED;
        for (int t = 1; t < a->buckets; ++t)
            if (a->bounds[t] <= a->bounds[t - 1]) return DLRM_ERR_INVALID_ARG;
    }
    if (a->d % 8 != 0 || a->d > 128 || a->Hq > 4096 || a->B >= (1 << 24)) return DLRM_ERR_UNSUPPORTED;
    if (a->Nq >= (int64_t(1) << 31) || a->Nkv >= (int64_t(1) << 31)) return DLRM_ERR_UNSUPPORTED;
    if (need_q_offsets) {  // a launch holds fewer than 2^32 work-items
        const int64_t most = (int64_t(1) << 32) / (a->d <= 64 ? 128 : 256) - kNumXcd;
        if (slot_count(a->Nq > a->Nkv ? a->Nq : a->Nkv, a->B, kQT) > most) return DLRM_ERR_UNSUPPORTED;
    }
    const uintptr_t ib = a->index_type == DLRM_INDEX_I32 ? 4 : 8;
    if (a->B > 0) {
        if (!a->kv_begin || !a->kv_end || !aligned(a->kv_begin, ib) || !aligned(a->kv_end, ib)) return DLRM_ERR_INVALID_ARG;
        if (need_q_offsets && (!a->q_offsets || !aligned(a->q_offsets, ib))) return DLRM_ERR_INVALID_ARG;
    }
    if ((a->Nq > 0 && !a->q) || (a->Nkv > 0 && (!a->k || !a->v))) return DLRM_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || (a->bias && !aligned(a->bias, 4)))
        return DLRM_ERR_INVALID_ARG;
    const int64_t strides[6] = {a->q_row, a->q_head, a->k_row, a->k_head, a->v_row, a->v_head};
    for (int64_t s : strides)
        if (s % 8 != 0 || s < a->d) return DLRM_ERR_INVALID_ARG;
    for (int i = 0; i < 6; i += 2)
        if (strides[i] >= (1 << 24)) return DLRM_ERR_UNSUPPORTED;  // a tile's rows are 32-bit offsets apart
    *out = Args{};
    out->q = a->q, out->k = a->k, out->v = a->v;
    out->q_row = a->q_row, out->q_head = a->q_head, out->k_row = a->k_row, out->k_head = a->k_head;
    out->v_row = a->v_row, out->v_head = a->v_head;
    out->q_off = a->q_offsets, out->kv_begin = a->kv_begin, out->kv_end = a->kv_end;
    out->Nq = a->Nq, out->Nkv = a->Nkv;
    out->B = static_cast<int32_t>(a->B), out->Hq = a->Hq, out->Hkv = a->Hkv, out->group = a->Hq / a->Hkv, out->d = a->d;
    out->idx32 = a->index_type == DLRM_INDEX_I32;
    constexpr int32_t kFar = 1 << 30;  // past every distance; keeps the kernels' differences in 32 bits
    out->window = a->window < kFar ? a->window : kFar;
    out->sinks = !a->window ? 0 : a->sinks < kFar ? a->sinks : kFar;
    out->scale = a->scale;
    out->bias = a->bias, out->buckets = a->bias ? a->buckets : 0;
    for (int t = 0; t < out->buckets; ++t) out->bounds[t] = a->bounds[t];
    out->last = out->buckets ? out->bounds[out->buckets - 1] : 0;
    return DLRM_OK;
}

namespace {

// DP: the head's width rounded up (the products run over DP columns, those from d on are zeros);
// LP: columns of a row in LDS.  WQ wavefronts of 32 queries each, by WK that share a tile's keys:
// each then takes one of its two halves, and their results are joined at the end.
template <int DP, int LP, int WQ, int WK, int OCC, int NEAR>
__global__ __launch_bounds__(WQ * WK * 64, OCC) void k_seq_attn_fwd(const Args a, uint16_t *o_out, float *lse_out,
                                                                    int32_t *tiles_out) {
    constexpr int QT = WQ * 32, STEPS = DP / 16, MB = DP / 32, THREADS = WQ * WK * 64;
    constexpr int TAB = QT + kBK, TILE = kBK * kPitch<LP>;
    __shared__ __attribute__((aligned(16))) uint16_t tiles_s[2 * TILE];
    __shared__ float near_s[kPad + NEAR], tab[TAB], bias_s[DLRM_SEQ_MAX_BUCKETS];
    __shared__ int bounds_s[DLRM_SEQ_MAX_BUCKETS];
    uint16_t *const Ks = tiles_s, *const Vs = tiles_s + TILE;

    const int slot = static_cast<int>(xcd_contiguous(blockIdx.x, gridDim.x));
    const int h = blockIdx.y;
    const int b = find_sequence(a, a.q_off, a.Nq, slot, QT);
    const Span sp = span_of(a, b);
    if (tiles_out && h == 0 && threadIdx.x == 0 && slot < slot_count(a.Nq, a.B, QT)) tiles_out[slot] = b;
    const int t = slot - (static_cast<int>(sp.q0) / QT + b);
    const int tiles = (sp.qlen + QT - 1) / QT;
    if (t < 0 || t >= tiles) return;
    const int q0 = (tiles - 1 - t) * QT;  // the last queries see the most keys: first

    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, half = lane >> 5;
    const int w = static_cast<int>(wave_id()) % WQ, wk = static_cast<int>(wave_id()) / WQ;
    const int kvh = h / a.group;
    const uint16_t *kb = a.k + sp.k0 * a.k_row + kvh * a.k_head;
    const uint16_t *vb = a.v + sp.k0 * a.v_row + kvh * a.v_head;

    // the keys that the block's queries see: [first, end), and the first `sinks`
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
    // Every query of the block sees every key of the tile at one bias: no table.
    const auto even = [&](int k0) {
        const int nearest = pmin - (k0 + kBK - 1);
        return nearest >= a.last && (!a.window || q0 + QT - 1 + sp.shift - k0 < a.window || k0 + kBK <= a.sinks);
    };
    const auto close = [&](int k0) { return pmin - k0 + QT - 1 < NEAR && k0 >= a.sinks; };
    const auto table = [&](int k0) {
        if (even(k0) || close(k0)) return;
        const int n0 = pmin - (k0 + kBK - 1);
        int bucket;
        for (int i = tid; i < TAB - 1; i += THREADS) tab[i] = bias_at(a, bounds_s, bias_s, n0 + i, k0 < a.sinks, &bucket);
    };

    // the queries, each lane's column of the second operand
    const int ql = q0 + w * 32 + ln;
    const bool live = ql < sp.qlen;
    Frag qf[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        qf[s].q = u32x4{0, 0, 0, 0};
        const int c = 16 * s + 8 * half;
        if (live && c < a.d)
            qf[s].q = *(const DLRM_GLOBAL u32x4 *)(a.q + (sp.q0 + ql) * a.q_row + h * a.q_head + c);
    }
    for (int i = tid; i < a.buckets; i += THREADS) {
        bounds_s[i] = a.bounds[i];
        bias_s[i] = a.bias[static_cast<int64_t>(h) * a.buckets + i];
    }

    __syncthreads();
    {
        const int reach = n > 0 ? min(NEAR, pmin + QT - t0 * kBK) : 0;  // past the furthest but for first keys'
        int bucket;
        for (int i = tid; i < reach; i += THREADS) near_s[kPad + i] = bias_at(a, bounds_s, bias_s, i, false, &bucket);
        for (int i = tid; i < kPad; i += THREADS) near_s[i] = -kInf;
    }

    f32x16 o[MB];
    float top, sum;
    const uint16_t *const krow = Ks + row_base<LP>(ln, half), *const vcol = Vs + column_base<LP>(lane);
    // One pass over the keys.  An infinity or NaN in a key would reach the queries that do not see it
    // (0 * NaN in a product): where a result is not finite, the block makes a second, WILD pass that keeps
    // the values apart.  What is finite makes no such pass, but pays for its code in registers: 207 with
    // it and 169 without at heads of 128, 128 and 120 at 64.  `start`: the reference that a pass
    // begins with; `share`: what a WILD one multiplies P by.
    const auto attend = [&](auto is_wild, float start, float share) {
        constexpr bool WILD = decltype(is_wild)::value;
#pragma unroll
        for (int m = 0; m < MB; ++m) o[m] = f32x16{};
        top = start, sum = 0.f;
        for (int it = 0; it < n; ++it) {
            const int k0 = key0(it);
            load(it);
            __syncthreads();  // the tile before has been read
            table(k0);
            ks.store(Ks);
            vs.store(Vs);
            __syncthreads();
            const int wpos = pmin + w * 32;  // position of the wavefront's first query
            // 32 keys at a time: S, P and their operands for 64 would cost a wavefront a SIMD
#pragma unroll 1
            for (int g = WK == 2 ? wk : 0; g < (WK == 2 ? wk + 1 : 2); ++g) {
                const int k1 = k0 + 32 * g;
                if (wpos + 31 < k1 || q0 + w * 32 >= sp.qlen || (a.window && wpos - (k1 + 31) >= a.window && k1 >= a.sinks))
                    continue;  // seen by none of the wavefront's queries
                const uint16_t *kt = krow + 32 * g * kPitch<LP>, *vt = vcol + 32 * g * kPitch<LP>;
                f32x16 s = f32x16{};
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    Frag k;
                    read_row(k, kt, i);
                    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k.b, qf[i].b, s, 0, 0, 0);
                }
                // register r: key 8 (r / 4) + 4 half + r % 4
                if (even(k0)) {
                    const float c = a.buckets ? bias_s[a.buckets - 1] : 0.f;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, c);
                } else {
                    // distance wpos + ln - k1 - 4 half - (key): entry 63 - that of tab's
                    const float *tb = close(k0) ? near_s + kPad + wpos - k1 + ln - 4 * half
                                                : tab + w * 32 + ln + kBK - 1 - 32 * g - 4 * half;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], a.scale, tb[-(8 * (r / 4) + r % 4)]);
                    if constexpr (WILD) {  // NaN - infinity is no -infinity
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (tb[-(8 * (r / 4) + r % 4)] == -kInf) s[r] = -kInf;
                    }
                    if (k0 < a.sinks) {
                        const int p = wpos + ln;
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int key = k1 + 8 * (r / 4) + 4 * half + r % 4;
                            if (p - key >= a.window && key >= a.sinks) s[r] = -kInf;
                        }
                    }
                }
                float mx = s[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[r]);
                mx = max_halves(mx);
                // the reference is moved when the maximum is over it by 8 (P up to e^8: bf16 holds that as well
                // as 1, and sums that it takes past the largest number are made again, below): with 32 rows one of them has a new maximum nearly every time
                const bool over = mx > top + 8.f;
                if (__any(over)) {
                    const float f = over ? __builtin_amdgcn_exp2f((top - mx) * kLog2e) : 1.f;
                    sum *= f;
#pragma unroll
                    for (int m = 0; m < MB; ++m)
#pragma unroll
                        for (int r = 0; r < 16; ++r) o[m][r] *= f;
                    top = over ? mx : top;
                }
                const float ref = top == -kInf ? 0.f : top;
                if (__any(fabsf(ref) > kHuge && fabsf(ref) < kInf)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f((s[r] - ref) * kLog2e);
                } else {
                    const float ref2 = ref * kLog2e;
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], kLog2e, -ref2));
                }
                if constexpr (WILD) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] *= share;
                }
                Frag p[2];
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    sum += s[r] + s[r + 1];
                    p[r / 8].w[r / 2 % 4] = pack_bf16(s[r], s[r + 1]);
                }
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        Frag v;
                        read_columns<LP>(v, vt, 16 * u, 32 * m);
                        if constexpr (WILD) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) v.w[e] = only_finite(v.w[e]);
                        }
                        o[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, p[u].b, o[m], 0, 0, 0);
                    }
                if constexpr (WILD) {
                    // the products above left out infinities and NaN; each kind reaches a query's output
                    // where the query sees such a key: counted by a product with the 0/1 visibility
                    const int p0 = wpos + ln;
                    Frag see[2];
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int key = k1 + 8 * (r / 4) + 4 * half + r % 4, dist = p0 - key;
                        const bool yes = dist >= 0 && (!a.window || dist < a.window || key < a.sinks);
                        const uint32_t bit = yes ? 0x3f80u : 0u;
                        uint32_t &word = see[r / 8].w[r / 2 % 4];
                        word = r % 2 ? word | bit << 16 : bit;
                    }
#pragma unroll 1
                    for (int kind = 0; kind < 3; ++kind) {
#pragma unroll
                        for (int m = 0; m < MB; ++m) {
                            f32x16 hit = f32x16{};
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                Frag v;
                                read_columns<LP>(v, vt, 16 * u, 32 * m);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    uint32_t out = 0;
#pragma unroll
                                    for (int k = 0; k < 2; ++k) {
                                        const uint32_t x = k ? v.w[e] >> 16 : v.w[e] & 0xffffu;
                                        const bool yes = kind == 0   ? x == 0x7f80u
                                                         : kind == 1 ? x == 0xff80u
                                                                     : (x & 0x7fffu) > 0x7f80u;
                                        out |= (yes ? 0x3f80u : 0u) << (16 * k);
                                    }
                                    v.w[e] = out;
                                }
                                hit = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, see[u].b, hit, 0, 0, 0);
                            }
                            const float add = kind == 0 ? kInf : kind == 1 ? -kInf : __builtin_nanf("");
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                if (hit[r] > 0.f) o[m][r] += add;
                        }
                    }
                }
            }
        }
        sum = add_halves(sum);
    };
    attend(std::false_type(), -kInf, 1.f);
    // An output is a mean of its values and finite where they are, but sum P v before the division may not be:
    // P adds up to as much as e^8 a key.  Where a query's o is still not finite after a WILD pass and its sum
    // is, a third pass takes that sum as known: P / sum adds up to 1.
    float unit = 1.f;  // of o, in the sum's terms
#pragma unroll 1
    for (int again = 0; again < 2; ++again) {
        float any = sum;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) any += o[m][r];
        const bool odd = !(fabsf(any) < kInf);
        const bool over = max_halves(odd && again == 1 && sum > 0.f && sum < kInf ? 1.f : 0.f) != 0.f;
        if (!__syncthreads_or(live && (again == 0 ? odd : over))) break;
        const float top0 = top, sum0 = sum;
        attend(std::true_type(), over ? top0 : -kInf, over ? 1.f / sum0 : 1.f);
        if (over) unit = sum0 / sum, top = top0, sum = sum0;
    }
    if constexpr (WK == 2) {  // the second half of the keys joins the first
        float *const part = reinterpret_cast<float *>(tiles_s) + w * (MB * 16 + 3) * 64 + lane;
        static_assert(WQ * (MB * 16 + 3) * 64 * 4 <= 2 * TILE * 2, "the tiles' room holds the halves' results");
        __syncthreads();
        if (wk == 1) {
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int r = 0; r < 16; ++r) part[(m * 16 + r) * 64] = o[m][r];
            part[MB * 16 * 64] = top;
            part[(MB * 16 + 1) * 64] = sum;
            part[(MB * 16 + 2) * 64] = unit;
        }
        __syncthreads();
        if (wk == 1) return;
        const float top1 = part[MB * 16 * 64], sum1 = part[(MB * 16 + 1) * 64], mx = fmaxf(top, top1);
        const float f0 = top == -kInf ? 0.f : top == mx ? 1.f : __builtin_amdgcn_exp2f((top - mx) * kLog2e);
        const float f1 = top1 == -kInf ? 0.f : top1 == mx ? 1.f : __builtin_amdgcn_exp2f((top1 - mx) * kLog2e);
        // a half without a key that the query sees holds a sum of 0; one whose every logit is NaN has the same
        // maximum, as that passes NaN over, and its sum is NaN
        sum = f0 * sum + f1 * sum1;
        top = mx;
        // divided before they are added: both may be near the largest number
        const float inv = sum == 0.f ? 0.f : 1.f / sum, g0 = f0 * unit * inv, g1 = f1 * part[(MB * 16 + 2) * 64] * inv;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[m][r] = g0 * o[m][r] + g1 * part[(m * 16 + r) * 64];
    }

    if (!live) return;
    const float inv = WK == 2 ? 1.f : sum == 0.f ? 0.f : unit / sum;
    const int64_t row = (sp.q0 + ql) * a.Hq + h;
    if (lse_out && half == 0) lse_out[row] = sum == 0.f ? -kInf : top + __builtin_amdgcn_logf(sum) * kLn2;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * m + 8 * g + 4 * half;
            if (c >= a.d) continue;
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = o[m][4 * g + r] * inv;
            const u32x2 hi = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
            *(DLRM_GLOBAL u32x2 *)(o_out + row * a.d + c) = hi;
        }
}

template <int DP, int LP, int WQ, int WK, int OCC, int NEAR>
int launch(const Args &a, uint16_t *o, float *lse, int32_t *tiles, hipStream_t stream) {
    const dim3 grid(round_up_xcd(slot_count(a.Nq, a.B, WQ * 32)), a.Hq);
    DLRM_LAUNCH("seq_attn_fwd", (k_seq_attn_fwd<DP, LP, WQ, WK, OCC, NEAR>), grid, dim3(WQ * WK * 64), 0, stream, a, o, lse, tiles);
    return launch_status();
}

}  // namespace
}  // namespace seq
}  // namespace dlrm

extern "C" size_t dlrm_seq_attn_tiles(int64_t B, int64_t Nq) {
    using namespace dlrm::seq;
    return B < 0 || B >= (1 << 24) || Nq < 0 || Nq >= (int64_t(1) << 31) ? 0 : slot_count(Nq, B, kQT);
}

extern "C" int dlrm_seq_attn_fwd(const dlrm_seq_attn *desc, uint16_t *o, float *lse, int32_t *tiles, dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq;
    Args a;
    const int rc = check_attn(desc, true, &a);
    if (rc != DLRM_OK) return rc;
    if (a.B > 0 && a.Nq > 0 && (lse == nullptr) != (tiles == nullptr)) return DLRM_ERR_INVALID_ARG;
    if (a.Nq > 0 && (!o || !aligned(o, 16) || !aligned(lse, 4) || !aligned(tiles, 4))) return DLRM_ERR_INVALID_ARG;
    if (a.B == 0 || a.Nq == 0) return DLRM_OK;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    // Wavefronts (queries x halves of a tile's keys) and their number a SIMD, at each width the best of
    // those tried.  Heads of 64: 2 x 1 took 78 us where 2 x 2 took 93 (the 1024 sequences above, before later
    // steps).  Of 128: 2 x 2 took 38 us where 4 x 1 took 50 and 2 x 1 with three a SIMD 53 (16 sequences of up
    // to 300 queries after up to 2048 keys).  The near biases: 2048 distances against 896 at heads of 32, 74 -> 70
    // us, and against 1280 at 128, 99 -> 97 (8 sequences of 2048, a bias that differs up to 2048); at 64 the
    // longer table costs a workgroup a CU: 86 -> 87, and 18.7 -> 20.5 for 64 sequences of 256.
    if (a.d <= 32) return launch<32, 32, 2, 1, 4, 2048>(a, o, lse, tiles, stream);
    if (a.d <= 64) return launch<64, 64, 2, 1, 4, 640>(a, o, lse, tiles, stream);
    return launch<128, 128, 2, 2, 2, 2048>(a, o, lse, tiles, stream);
}
