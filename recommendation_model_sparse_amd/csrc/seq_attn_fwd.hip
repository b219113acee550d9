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
// transposing LDS loads.
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
    if (a->Nq >= (int64_t(1) << 40) || a->Nkv >= (int64_t(1) << 40)) return DLRM_ERR_UNSUPPORTED;
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
    out->scale = a->scale, out->scale_log2 = a->scale * kLog2e;
    out->bias = a->bias, out->buckets = a->bias ? a->buckets : 0;
    for (int t = 0; t < out->buckets; ++t) out->bounds[t] = a->bounds[t];
    out->last = out->buckets ? out->bounds[out->buckets - 1] : 0;
    return DLRM_OK;
}

namespace {

// DP: the head's width rounded up (the products run over DP columns, those from d on are zeros);
// LP: columns of a row in LDS; NW: wavefronts of 32 queries.
template <int DP, int LP, int NW, bool TRAIN>
__global__ __launch_bounds__(NW * 64) void k_seq_attn_fwd(const Args a, uint16_t *o_out, float *lo_out, float *lse_out,
                                                          const int64_t slots) {
    constexpr int QT = NW * 32, STEPS = DP / 16, MB = DP / 32, THREADS = NW * 64;
    constexpr int TAB = QT + kBK;
    __shared__ __attribute__((aligned(16))) uint16_t Ks[2][kBK * LP], Vs[2][kBK * LP];
    __shared__ float tab[2][TAB], bias_s[DLRM_SEQ_MAX_BUCKETS];
    __shared__ int bounds_s[DLRM_SEQ_MAX_BUCKETS];

    const int64_t id = xcd_contiguous(blockIdx.x, gridDim.x);
    if (id >= slots * a.Hq) return;
    const int h = static_cast<int>(id / slots);
    const int64_t slot = id - h * slots;
    const int b = find_sequence(a, a.q_off, a.Nq, slot, QT);
    const Span sp = span_of(a, b);
    const int64_t t = slot - (sp.q0 / QT + b);
    const int tiles = (sp.qlen + QT - 1) / QT;
    if (t < 0 || t >= tiles) return;
    const int q0 = (tiles - 1 - static_cast<int>(t)) * QT;  // the last queries see the most keys: first

    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, half = lane >> 5;
    const int w = static_cast<int>(wave_id());
    const int kvh = h / a.group;
    const uint16_t *kb = a.k + sp.k0 * a.k_row + kvh * a.k_head;
    const uint16_t *vb = a.v + sp.k0 * a.v_row + kvh * a.v_head;

    for (int i = tid; i < a.buckets; i += THREADS) {
        bounds_s[i] = a.bounds[i];
        bias_s[i] = a.bias[static_cast<int64_t>(h) * a.buckets + i];
    }

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

    // the keys that the block's queries see: [first, end), and the first `sinks`
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
    // Every query of the block sees every key of the tile / at one bias.
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
            int bucket;
            for (int i = tid; i < TAB - 1; i += THREADS)
                tab[buf][i] = table_entry(a, bounds_s, bias_s, n0 + i, k0 < a.sinks, &bucket);
        }
    };

    f32x16 o[MB];
    float top, sum;
    // One pass over the keys.  An infinity or NaN in a key would reach the queries that do not see it
    // (0 * NaN in a product): where a result is NaN, the block makes a second, WILD pass that keeps
    // the values apart.  What is finite pays nothing for it.
    const auto attend = [&](auto is_wild) {
    constexpr bool WILD = decltype(is_wild)::value;
#pragma unroll
    for (int m = 0; m < MB; ++m) o[m] = f32x16{};
    top = -kInf, sum = 0.f;
    if (n > 0) load(0);
    __syncthreads();
    if (n > 0) fill(0);
    for (int it = 0; it < n; ++it) {
        const int k0 = key0(it), buf = it & 1;
        if (it + 1 < n) load(it + 1);
        __syncthreads();
        const int wpos = pmin + w * 32;  // position of the wavefront's first query
        const bool none = wpos + 31 < k0 || q0 + w * 32 >= sp.qlen ||
                          (a.window && wpos - (k0 + kBK - 1) >= a.window && k0 >= a.sinks);
        if (!none) {
            f32x16 s[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                s[g] = f32x16{};
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    Frag k;
                    read_row<LP>(k, Ks[buf], 32 * g + ln, 2 * i + half);
                    s[g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k.b, qf[i].b, s[g], 0, 0, 0);
                }
            }
            // register r of block g: key 32 g + 8 (r / 4) + 4 half + r % 4
            if (even(k0)) {
                const float c = a.buckets ? bias_s[a.buckets - 1] : 0.f;
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[g][r] = fmaf(s[g][r], a.scale, c);
            } else {
                const float *tb = tab[buf] + w * 32 + ln + kBK - 1 - 4 * half;
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[g][r] = fmaf(s[g][r], a.scale, tb[-(32 * g + 8 * (r / 4) + r % 4)]);
                if constexpr (WILD) {  // NaN - infinity is no -infinity
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (tb[-(32 * g + 8 * (r / 4) + r % 4)] == -kInf) s[g][r] = -kInf;
                }
                if (k0 < a.sinks) {
                    const int p = wpos + ln;
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int key = k0 + 32 * g + 8 * (r / 4) + 4 * half + r % 4;
                            if (p - key >= a.window && key >= a.sinks) s[g][r] = -kInf;
                        }
                }
            }
            float mx = s[0][0];
#pragma unroll
            for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[0][r]);
#pragma unroll
            for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[1][r]);
            mx = fmaxf(max_halves(mx), top);
            if (__any(mx > top)) {
                const float f = mx == -kInf ? 1.f : __builtin_amdgcn_exp2f((top - mx) * kLog2e);
                sum *= f;
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[m][r] *= f;
                top = mx;
            }
            const float ref = top == -kInf ? 0.f : top;
            if (__any(fabsf(ref) > kHuge && fabsf(ref) < kInf)) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[g][r] = __builtin_amdgcn_exp2f((s[g][r] - ref) * kLog2e);
            } else {
                const float ref2 = ref * kLog2e;
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[g][r] = __builtin_amdgcn_exp2f(fmaf(s[g][r], kLog2e, -ref2));
            }
            Frag p[2][2], p_mid[2][2], p_lo[2][2];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    sum += s[g][r] + s[g][r + 1];
                    const uint32_t hi = pack_bf16(s[g][r], s[g][r + 1]);
                    p[g][r / 8].w[r / 2 % 4] = hi;
                    if constexpr (TRAIN) {  // all 24 bits of P, in three pieces
                        const float x = s[g][r] - bf16_lo(hi), y = s[g][r + 1] - bf16_hi(hi);
                        const uint32_t mid = pack_bf16(x, y);
                        p_mid[g][r / 8].w[r / 2 % 4] = mid;
                        p_lo[g][r / 8].w[r / 2 % 4] = pack_bf16(x - bf16_lo(mid), y - bf16_hi(mid));
                    }
                }
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        Frag v;
                        read_columns<LP>(v, Vs[buf], 32 * g + 16 * u, 32 * m, lane);
                        if constexpr (WILD) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) v.w[e] = only_finite(v.w[e]);
                        }
                        o[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, p[g][u].b, o[m], 0, 0, 0);
                        if constexpr (TRAIN) {
                            o[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, p_mid[g][u].b, o[m], 0, 0, 0);
                            o[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, p_lo[g][u].b, o[m], 0, 0, 0);
                        }
                    }
            if constexpr (WILD) {
                // the products above left out infinities and NaN; each kind reaches a query's output
                // where the query sees such a key: counted by a product with the 0/1 visibility
                const int p0 = wpos + ln;
                Frag see[2][2];
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int key = k0 + 32 * g + 8 * (r / 4) + 4 * half + r % 4, dist = p0 - key;
                        const bool yes = dist >= 0 && (!a.window || dist < a.window || key < a.sinks);
                        const uint32_t bit = yes ? 0x3f80u : 0u;
                        uint32_t &word = see[g][r / 8].w[r / 2 % 4];
                        word = r % 2 ? word | bit << 16 : bit;
                    }
#pragma unroll 1
                for (int kind = 0; kind < 3; ++kind) {
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        f32x16 hit = f32x16{};
#pragma unroll
                        for (int g = 0; g < 2; ++g)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                Frag v;
                                read_columns<LP>(v, Vs[buf], 32 * g + 16 * u, 32 * m, lane);
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
                                hit = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, see[g][u].b, hit, 0, 0, 0);
                            }
                        const float add = kind == 0 ? kInf : kind == 1 ? -kInf : __builtin_nanf("");
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (hit[r] > 0.f) o[m][r] += add;
                    }
                }
            }
        }
        if (it + 1 < n) fill(it + 1);  // its buffer was last read before this tile's barrier
    }
    sum = add_halves(sum);
    };
    attend(std::false_type());
    float any = sum;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) any += o[m][r];
    if (__syncthreads_or(live && any != any)) attend(std::true_type());

    if (!live) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t row = (sp.q0 + ql) * a.Hq + h;
    if constexpr (TRAIN) {
        if (half == 0) lse_out[row] = sum == 0.f ? -kInf : top + __builtin_amdgcn_logf(sum) * kLn2;
    }
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
            if constexpr (TRAIN) {
                *(DLRM_GLOBAL floatx4 *)(lo_out + row * a.d + c) = floatx4{x[0] - bf16_lo(hi.x), x[1] - bf16_hi(hi.x),
                                                                          x[2] - bf16_lo(hi.y), x[3] - bf16_hi(hi.y)};
            }
        }
}

template <int DP, int LP, int NW>
int launch(const Args &a, uint16_t *o, float *o_lo, float *lse, hipStream_t stream) {
    const int64_t slots = slot_count(a.Nq, a.B, NW * 32);
    const int64_t blocks = slots * a.Hq;
    if (blocks >= (int64_t(1) << 31) - 8) return DLRM_ERR_UNSUPPORTED;
    const dim3 grid(round_up_xcd(blocks)), block(NW * 64);
    if (lse)
        DLRM_LAUNCH("seq_attn_fwd_train", (k_seq_attn_fwd<DP, LP, NW, true>), grid, block, 0, stream, a, o, o_lo, lse, slots);
    else
        DLRM_LAUNCH("seq_attn_fwd", (k_seq_attn_fwd<DP, LP, NW, false>), grid, block, 0, stream, a, o, o_lo, lse, slots);
    return launch_status();
}

}  // namespace
}  // namespace seq
}  // namespace dlrm

extern "C" int dlrm_seq_attn_fwd(const dlrm_seq_attn *desc, uint16_t *o, float *o_lo, float *lse,
                                 dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq;
    Args a;
    const int rc = check_attn(desc, true, &a);
    if (rc != DLRM_OK) return rc;
    if ((o_lo == nullptr) != (lse == nullptr)) return DLRM_ERR_INVALID_ARG;
    if (a.Nq > 0 && (!o || !aligned(o, 16) || !aligned(o_lo, 16) || !aligned(lse, 4))) return DLRM_ERR_INVALID_ARG;
    if (a.B == 0 || a.Nq == 0) return DLRM_OK;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    if (a.d <= 32) return launch<32, 32, 4>(a, o, o_lo, lse, stream);
    if (a.d <= 64) return launch<64, 64, 4>(a, o, o_lo, lse, stream);
    return launch<128, 128, 4>(a, o, o_lo, lse, stream);
}
