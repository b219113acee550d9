// Shared by the kernels of linear attention with a decay (dlrm_seq_decay.h).
//
// Everything is one operation on rows x, y and z, forward or in reverse time:
//
//     out_i = scale sum_{j seen by i} w_ij <x_i, y_j> z_j
//
// the output from (q, k, v), dq from (do, v, k), and in reverse, where i sees the events after it,
// dk from (v, do, q) and dv from (k, q, do).  It is worked out in chunks of 64 events: pairs within a
// chunk as products of tiles, everything before through a state, S = sum_j w_j y_j z_j^T.  With G the sums
// of g from the chunk's first event on, and n its last:
//
//     out_i = scale (e^{G_i} S^T x_i + sum_{j<=i} e^{G_i - G_j} <x_i, y_j> z_j);   S <- e^{G_n} S + sum_j e^{G_n - G_j} y_j z_j^T
//
// and in reverse e^{G_n - G_j} on the way out and e^{G_i} on the way in.
//
// A workgroup walks the chunks of one sequence and key head.  Each of its LP / 32 wavefronts has 32
// columns of the state in its accumulators (32x32x16 matrix instructions: rows of y, columns of z), and
// those columns of the outputs, as transposed tiles: out^T = S^T x^T + z^T P^T.  The state's accumulators are,
// rounded, the first operand as they stand; P^T goes through LDS, as every wavefront needs all of it.
#pragma once

#include "dlrm_seq_decay.h"
#include "seq.h"

namespace dlrm {
namespace seq {
namespace decay {

constexpr int kC = 64;    // events of a chunk
constexpr int kPP = 72;   // elements from one row of P to the next
constexpr float kLeast = -104.f;  // e^-104 is 0 in fp32: decays below are taken as it, so that sums stay finite

struct Heads {  // [rows][heads][d] bf16
    const uint16_t *p;
    int64_t row, head;
};

struct Walk {
    Heads x, y, z, t;  // t: what the gradient of the decays takes beside them
    const float *g;
    int64_t g_row;
    const void *off;
    int64_t N;
    int32_t idx32, B, Hq, Hkv, group, d;
    float scale;
    int32_t run;         // chunks of a run, a workgroup's share of a sequence; 0: the whole of it
    uint32_t slots;      // runs, or sequences
    const float *start;  // states: of runs [slots][Hkv][d][d], or [B][Hkv][d][d]; NULL: zeros
    float *last;         // [B][Hkv][d][d] or NULL
    float *fade;         // e^(sum of g) of each run, [slots][Hkv]
    uint16_t *out, *out2;
    float *terms;  // [Hkv][N]
};

// Which chunks of which sequence a workgroup walks.
struct Part {
    int64_t row0;
    int b, len, chunks, c0, c1, kvh;
    uint32_t slot;
    bool any;
};

__device__ __forceinline__ Part part_of(const Walk &a, uint32_t id) {
    Part p;
    p.slot = id / static_cast<uint32_t>(a.Hkv), p.kvh = static_cast<int>(id - p.slot * a.Hkv);
    p.any = p.slot < a.slots;
    if (!p.any) return p;
    const int T = kC * a.run;
    p.b = a.run ? find_sequence(a, a.off, a.N, static_cast<int>(p.slot), T) : static_cast<int>(p.slot);
    const int r0 = offset_at(a, a.off, p.b, a.N), r1 = offset_at(a, a.off, p.b + 1, a.N);
    p.row0 = r0, p.len = max(r1 - r0, 0);
    p.chunks = (p.len + kC - 1) / kC;
    const int r = a.run ? static_cast<int>(p.slot) - (r0 / T + p.b) : 0;
    p.c0 = r * a.run;
    p.c1 = a.run ? min(p.c0 + a.run, p.chunks) : p.chunks;
    p.any = r >= 0 && (r == 0 || p.c0 < p.chunks);
    return p;
}

// What a chunk's decays come to, for each event: its sum G as two fp32 numbers (their sum holds 48 bits:
// differences are exact to fp32 whatever pauses lie between), e^G and e^{G_n - G}, in base 2.
struct Decays {
    float hi[kC], lo[kC], from[kC], to[kC];
};

__device__ __forceinline__ float decay_load(const Walk &a, const Part &p, int c, int lane) {
    const int i = c * kC + lane;
    return i < p.len ? a.g[(p.row0 + i) * a.g_row + p.kvh] : 0.f;
}

// By one wavefront, lane = event; returns e^{G_n} to all lanes and adds G_n to *total.
__device__ __forceinline__ float decays(Decays &out, float g, int lane, double *total) {
    g = g > 0.f ? 0.f : g < kLeast ? kLeast : g;  // NaN stays
    double s = static_cast<double>(g) * 1.4426950408889634;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
        const double up = __shfl_up(s, i);
        if (lane >= i) s += up;
    }
    const double n = __shfl(s, 63);
    *total += n;
    const float hi = static_cast<float>(s);
    out.hi[lane] = hi;
    out.lo[lane] = static_cast<float>(s - hi);
    out.from[lane] = __builtin_amdgcn_exp2f(hi);
    out.to[lane] = __builtin_amdgcn_exp2f(static_cast<float>(n - s));
    return __builtin_amdgcn_exp2f(static_cast<float>(n));
}

template <int LP>
struct Of {
    static constexpr int WAVES = LP / 32, CT = LP / 32, STEPS = LP / 16, TILE = kC * kPitch<LP>;
};

// The high halves of two words.
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Eight fp32 values as N bf16 operands that add up to them: 1 rounded to nearest, 2 to 2^-17, 3 exactly
// (8 bits of the 24 at a time, cut off).
template <int N>
__device__ __forceinline__ void parts_of(const float (&x)[8], Frag (&out)[N]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float a = x[e], b = x[e + 1];
        if constexpr (N == 1) {
            out[0].w[e / 2] = pack_bf16(a, b);
        } else if constexpr (N == 2) {
            const uint32_t hi = pack_bf16(a, b);
            out[0].w[e / 2] = hi;
            out[1].w[e / 2] = pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
        } else {
            const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
            const float ra = a - bf16_hi(ua), rb = b - bf16_hi(ub);
            const uint32_t va = __float_as_uint(ra), vb = __float_as_uint(rb);
            const float sa = ra - bf16_hi(va), sb = rb - bf16_hi(vb);
            out[0].w[e / 2] = high_halves(ua, ub);
            out[1].w[e / 2] = high_halves(va, vb);
            out[2].w[e / 2] = high_halves(__float_as_uint(sa), __float_as_uint(sb));
        }
    }
}

// S from memory (rows y, columns z; TRANSPOSED: the other way round) or zeros.
template <int LP, bool TRANSPOSED>
__device__ __forceinline__ void state_load(f32x16 (&S)[Of<LP>::CT], const float *p, int d, int w, int lane) {
    const int ln = lane & 31, half = lane >> 5, e = 32 * w + ln;
#pragma unroll
    for (int ct = 0; ct < Of<LP>::CT; ++ct) S[ct] = f32x16{};
    if (!p || e >= d) return;
#pragma unroll
    for (int ct = 0; ct < Of<LP>::CT; ++ct)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (32 * ct + 8 * k >= d) continue;  // d is a multiple of 8
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int c = 32 * ct + 8 * k + 4 * half + r;
                S[ct][4 * k + r] = p[TRANSPOSED ? e * d + c : c * d + e];
            }
        }
}

template <int LP>
__device__ __forceinline__ void state_store(const f32x16 (&S)[Of<LP>::CT], float *p, int d, int w, int lane) {
    const int ln = lane & 31, half = lane >> 5, e = 32 * w + ln;
    if (e >= d) return;
#pragma unroll
    for (int ct = 0; ct < Of<LP>::CT; ++ct)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (32 * ct + 8 * k >= d) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) p[(32 * ct + 8 * k + 4 * half + r) * d + e] = S[ct][4 * k + r];
        }
}

// S <- fade S + sum_j w_j y_j z_j^T
template <int LP, int UP>
__device__ __forceinline__ void state_grow(f32x16 (&S)[Of<LP>::CT], const uint16_t *ys, const uint16_t *zs, const float *weight, int w,
                                           int lane) {
    const uint16_t *ycol = ys + column_base<LP>(lane), *zcol = zs + column_base<LP>(lane);
    const int half = lane >> 5;
#pragma unroll
    for (int u = 0; u < kC / 16; ++u) {
        Frag z, zw[UP];
        read_columns<LP>(z, zcol, 16 * u, 32 * w);
        const floatx4 w0 = *reinterpret_cast<const floatx4 *>(weight + 16 * u + 4 * half);
        const floatx4 w1 = *reinterpret_cast<const floatx4 *>(weight + 16 * u + 8 + 4 * half);
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = bf16_lo(z.w[e]) * (e < 2 ? w0[2 * e % 4] : w1[2 * e % 4]);
            x[2 * e + 1] = bf16_hi(z.w[e]) * (e < 2 ? w0[2 * e % 4 + 1] : w1[2 * e % 4 + 1]);
        }
        parts_of<UP>(x, zw);
#pragma unroll
        for (int ct = 0; ct < Of<LP>::CT; ++ct) {
            Frag y;
            read_columns<LP>(y, ycol, 16 * u, 32 * ct);
#pragma unroll
            for (int n = 0; n < UP; ++n) S[ct] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y.b, zw[n].b, S[ct], 0, 0, 0);
        }
    }
}

// A lane's eight values of row `row`, columns 16 s + 4 half + {0..3} and those 8 further on: the order of an
// accumulator's rows.
template <int LP>
__device__ __forceinline__ void read_row_as_rows(Frag &f, const uint16_t *tile, int row, int half, int s) {
    const uint16_t *at = tile + row * kPitch<LP> + 4 * half + 16 * s;
    const u32x2 a = *reinterpret_cast<const u32x2 *>(at), b = *reinterpret_cast<const u32x2 *>(at + 8);
    f.w[0] = a.x, f.w[1] = a.y, f.w[2] = b.x, f.w[3] = b.y;
}

// o^T = S^T x^T for both halves of the chunk's rows.
template <int LP, int PR>
__device__ __forceinline__ void through_state(f32x16 (&o)[2], const f32x16 (&S)[Of<LP>::CT], const uint16_t *xs, int lane) {
    const int ln = lane & 31, half = lane >> 5;
    o[0] = o[1] = f32x16{};
#pragma unroll
    for (int s = 0; s < Of<LP>::STEPS; ++s) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = S[s / 2][8 * (s % 2) + e];
        Frag f[PR];
        parts_of<PR>(v, f);
#pragma unroll
        for (int ib = 0; ib < 2; ++ib) {
            Frag x;
            read_row_as_rows<LP>(x, xs, 32 * ib + ln, half, s);
#pragma unroll
            for (int n = 0; n < PR; ++n) o[ib] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[n].b, x.b, o[ib], 0, 0, 0);
        }
    }
}

// Tile t of the three that hold pairs that see each other: rows jb of y, ib of x.
template <bool REV>
__device__ __forceinline__ void tile_of(int t, int *jb, int *ib) {
    *ib = REV ? t == 2 : t > 0;
    *jb = REV ? t > 0 : t == 2;
}

// P^T = <y_j, x_i> e^{..}, rounded to bf16, one tile, to LDS: row i, its j in the order of an operand's
// lanes.  MORE: also sums over j of P times the product of a second pair of rows, for each i (kept unrounded: the
// decays' gradient is fp32); x2(s) gives a lane's share of the second x at step s.
template <int LP, bool REV, bool MORE, typename X2>
__device__ __forceinline__ float pair_tile(uint16_t *P, const Decays &dec, const uint16_t *xs, const uint16_t *ys, X2 x2,
                                           const uint16_t *y2s, int jb, int ib, int lane) {
    const int ln = lane & 31, half = lane >> 5;
    f32x16 s = f32x16{}, m = f32x16{};
#pragma unroll
    for (int i = 0; i < Of<LP>::STEPS; ++i) {
        Frag x, y;
        read_row(x, xs + row_base<LP>(32 * ib + ln, half), i);
        read_row(y, ys + row_base<LP>(32 * jb + ln, half), i);
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y.b, x.b, s, 0, 0, 0);
        if constexpr (MORE) {
            const Frag u = x2(i);
            Frag v;
            read_row(v, y2s + row_base<LP>(32 * jb + ln, half), i);
            m = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.b, u.b, m, 0, 0, 0);
        }
    }
    const int i = 32 * ib + ln;
    const float hi = dec.hi[i], lo = dec.lo[i];
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int j0 = 32 * jb + 8 * g + 4 * half;
        const floatx4 hj = *reinterpret_cast<const floatx4 *>(dec.hi + j0), lj = *reinterpret_cast<const floatx4 *>(dec.lo + j0);
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float diff = REV ? (hj[r] - hi) + (lj[r] - lo) : (hi - hj[r]) + (lo - lj[r]);
            const bool sees = REV ? j0 + r >= i : j0 + r <= i;
            const float x = s[4 * g + r] * __builtin_amdgcn_exp2f(diff);
            p[r] = sees ? x : 0.f;
            if constexpr (MORE) sum += sees ? x * m[4 * g + r] : 0.f;
        }
        *reinterpret_cast<u32x2 *>(P + i * kPP + 32 * jb + 16 * (g / 2) + 8 * half + 4 * (g % 2)) =
            u32x2{pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3])};
    }
    return MORE ? add_halves(sum) : 0.f;
}

// o^T += z^T P^T
template <int LP, bool REV>
__device__ __forceinline__ void through_pairs(f32x16 (&o)[2], const uint16_t *P, const uint16_t *zs, int w, int lane) {
    const uint16_t *zcol = zs + column_base<LP>(lane);
    const uint16_t *row = P + (lane & 31) * kPP + 8 * (lane >> 5);
#pragma unroll
    for (int u = 0; u < kC / 16; ++u) {
        Frag z;
        read_columns<LP>(z, zcol, 16 * u, 32 * w);
#pragma unroll
        for (int ib = 0; ib < 2; ++ib) {
            if (REV ? ib == 1 && u < 2 : ib == 0 && u >= 2) continue;  // none of its pairs see each other
            Frag p;
            p.q = *reinterpret_cast<const u32x4 *>(row + 32 * ib * kPP + 16 * u);
            o[ib] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(z.b, p.b, o[ib], 0, 0, 0);
        }
    }
}

// The same one row of z at a time, added where it is seen: what a row after it holds does not reach an output,
// though 0 * infinity is NaN.
template <int LP>
__device__ __forceinline__ void through_pairs_apart(f32x16 (&o)[2], const uint16_t *P, const uint16_t *zs, int w, int lane) {
    const uint16_t *zcol = zs + column_base<LP>(lane);
    const uint16_t *row = P + (lane & 31) * kPP + 8 * (lane >> 5);
#pragma unroll 1
    for (int j = 0; j < kC; ++j) {
        const int u = j / 16, mine = j % 16 - 4 * (lane >> 5);  // which of a lane's rows 0..3 and 8..11
        Frag z;
        read_columns<LP>(z, zcol, 16 * u, 32 * w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int first = 8 * (e / 2) + 2 * (e % 2);
            z.w[e] = mine == first ? z.w[e] & 0xffffu : mine == first + 1 ? z.w[e] & 0xffff0000u : 0u;
        }
#pragma unroll
        for (int ib = 0; ib < 2; ++ib) {
            Frag p;
            p.q = *reinterpret_cast<const u32x4 *>(row + 32 * ib * kPP + 16 * u);
            if (j > 32 * ib + (lane & 31)) p.q = u32x4{0, 0, 0, 0};  // the tile that nobody sees is not written
            const f32x16 add = __builtin_amdgcn_mfma_f32_32x32x16_bf16(z.b, p.b, f32x16{}, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (j <= 32 * ib + (lane & 31)) o[ib][r] += add[r];
        }
    }
}

// Rows of one chunk's outputs, columns 32 w on.
template <int LP>
__device__ __forceinline__ void out_rows(const f32x16 (&o)[2], uint16_t *out, int64_t stride, int rows, int d, float scale, int w,
                                         int lane) {
    const int ln = lane & 31, half = lane >> 5;
#pragma unroll
    for (int ib = 0; ib < 2; ++ib) {
        if (32 * ib + ln >= rows) continue;
        uint16_t *at = out + (32 * ib + ln) * stride;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = 32 * w + 8 * g + 4 * half;
            if (32 * w + 8 * g < d)
                *(DLRM_GLOBAL u32x2 *)(at + c) = u32x2{pack_bf16(o[ib][4 * g] * scale, o[ib][4 * g + 1] * scale),
                                                       pack_bf16(o[ib][4 * g + 2] * scale, o[ib][4 * g + 3] * scale)};
        }
    }
}

// ---------------------------------------------------------------- host

// Checks the description and fills what all walks share.
int check(const dlrm_seq_decay *a, bool offsets, Walk *out);

// How sequences are cut: chunks of a run (0: not), and the workgroups' places.
struct Cut {
    int32_t run;
    int64_t slots;
};
Cut cut_of(const Walk &a, int64_t max_len);

int64_t state_floats(const Walk &a, const Cut &c);  // of the runs' states and fades

// The states at the start of every run, forward (y and z of `a`) or reversed, into `states`.
// `first`: what sequences begin with, or NULL.
int run_states(const Walk &a, const Cut &c, bool reversed, int up, const float *first, float *states, hipStream_t stream);

// The forward walk; `up` and `more` as the kernel's.
int walk(const Walk &a, int up, bool more, hipStream_t stream);

}  // namespace decay
}  // namespace seq
}  // namespace dlrm
