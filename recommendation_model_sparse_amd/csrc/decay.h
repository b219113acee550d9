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
// A workgroup walks the chunks of one sequence and key head.  Each of its LP / 16 wavefronts has 16 columns of
// the state in its accumulators (16x16x32 matrix instructions: rows of y, columns of z), and those columns of the
// outputs, as transposed tiles: out^T = S^T x^T + z^T P^T.  The state's accumulators are, rounded, the first operand
// as they stand; P^T goes through LDS, as every wavefront needs all of it.  (With 32 columns a wavefront, on
// 32x32x16, half as many wavefronts waited twice as long: a chunk of heads of 128 took 8100 cycles of a workgroup
// by itself, of 64 7200.)
//
// Pairs' weights, and states on their way to an output, are rounded to bf16, as the matrix instructions take it (three parts
// of a weight would be three products): outputs are 2.3e-3 from the formula in 64 bits, of which their own rounding is 1.6e-3.
//
// A chunk takes 64 d (64 + 2 d) multiply-adds a head, so the rows' bytes are the floor: 291 MB forward and backward for 1024
// sequences of 16 to 512, 2 heads of 64, 60 us at the rate of a large copy.  The two calls take 183 us.  Their kernels, by the
// profiler, under which they take longer: o 38 (3.8 TB/s), dq 61, dk and dv 94, with a gradient of each event's decay, and
// twice 5 for the order, 203.  There the VALU is busy for half of the time (states split into bf16 parts, pairs weighed and
// packed, and scalar registers spilled to its own: 56 to 87 in the forward walks, 32 to 44 in those back with dg), LDS for 34 to
// 43 %, the matrix instructions for 11 to 18 %, at 2.3 to 2.9 wavefronts a SIMD.  4 sequences of 2000 to 4096, 8 heads of 128 over 2,
// take 167, by the profiler 173 of which 47 are the states at the runs' starts; the walks have one or two workgroups a CU there and
// wait for their own barriers.
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
    int32_t splits;      // workgroups that share a group's query heads (forward)
    uint32_t slots;      // runs, or sequences
    const int32_t *order;  // [B] the sequences, those of the most chunks first; NULL: as they come
    const float *first;  // what sequences begin with, [B][Hkv][d][d], or NULL: zeros
    float *start;        // the states at the start of the runs after a sequence's first, [slots][Hkv][d][d]
    bool all_start;      // and of its first: `last` is `first`, which other workgroups may write before one has read it
    float *last;         // [B][Hkv][d][d] or NULL
    float *fade;         // e^(sum of g) of each run, [slots][Hkv]
    uint16_t *out, *out2;
    // for the decays' gradient
    float *terms;        // [parts][Hkv][N]: <t, out> of the walk for dq, for each of its splits, by way of the state
    float *pairs;        // and by way of the chunk's pairs
    int32_t parts;
    float *marks;        // the forward state (dq's) before every `mark`th chunk but the first, as its wavefronts hold it (mark_at)
    int32_t mark;
    float *dg;           // [N][Hkv]
    double *sums;        // or over each slot's events, [Hkv][slots]
};

// Which chunks of which sequence a workgroup walks, and for which query heads of a group.
struct Part {
    int64_t row0;
    int b, len, chunks, c0, c1, kvh, split;
    uint32_t slot;
    bool any;
};

// A slot's workgroups, which read the same rows, go to one XCD, and the slots to the XCDs in turn.
__device__ __forceinline__ Part part_of(const Walk &a) {
    Part p;
    const uint32_t of_slot = a.Hkv * a.splits, turn = blockIdx.x / (kNumXcd * of_slot), at = blockIdx.x - turn * kNumXcd * of_slot;
    const uint32_t id = (turn * kNumXcd + at % kNumXcd) * of_slot + at / kNumXcd;
    const uint32_t one = id / static_cast<uint32_t>(a.splits);
    p.split = static_cast<int>(id - one * a.splits);
    p.slot = one / static_cast<uint32_t>(a.Hkv), p.kvh = static_cast<int>(one - p.slot * a.Hkv);
    p.any = p.slot < a.slots;
    if (!p.any) return p;
    const int T = kC * a.run;
    p.b = a.run ? find_sequence(a, a.off, a.N, static_cast<int>(p.slot), T) : a.order ? a.order[p.slot] : static_cast<int>(p.slot);
    const int r0 = offset_at(a, a.off, p.b, a.N), r1 = offset_at(a, a.off, p.b + 1, a.N);
    p.row0 = r0, p.len = max(r1 - r0, 0);
    p.chunks = (p.len + kC - 1) / kC;
    const int r = a.run ? static_cast<int>(p.slot) - (r0 / T + p.b) : 0;
    p.c0 = r * a.run;
    p.c1 = a.run ? min(p.c0 + a.run, p.chunks) : p.chunks;
    p.any = r >= 0 && (r == 0 || p.c0 < p.chunks);
    return p;
}

// The place of the state before chunk c > 0, a multiple of `mark`.  c / mark whole marks of the sequence's rows lie before it, so
// that no two sequences meet in a place, and N / (64 mark) places a key head are enough however many sequences there are.
__device__ __forceinline__ int64_t mark_at(const Walk &a, const Part &p, int c) {
    return (p.row0 / (kC * a.mark) + c / a.mark - 1) * a.Hkv + p.kvh;
}

// A sum over the lanes up to each, in fp64.
template <int CTRL, int ROWS>
__device__ __forceinline__ double from_lanes_below(double x) {
    const int64_t v = __double_as_longlong(x);
    const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), CTRL, ROWS, 0xf, false);
    return __longlong_as_double(static_cast<int64_t>(hi) << 32 | static_cast<uint32_t>(lo));
}
__device__ __forceinline__ double prefix_sum(double s) {
    s += from_lanes_below<0x111, 0xf>(s);  // the lane 1, 2, 4, 8 below, within 16
    s += from_lanes_below<0x112, 0xf>(s);
    s += from_lanes_below<0x114, 0xf>(s);
    s += from_lanes_below<0x118, 0xf>(s);
    s += from_lanes_below<0x142, 0xa>(s);  // the last of the 16 below; of the 32 below
    s += from_lanes_below<0x143, 0xc>(s);
    return s;
}
__device__ __forceinline__ double last_lane(double x) {
    const int64_t v = __double_as_longlong(x);
    const int lo = __builtin_amdgcn_readlane(static_cast<int>(v), 63), hi = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), 63);
    return __longlong_as_double(static_cast<int64_t>(hi) << 32 | static_cast<uint32_t>(lo));
}

// What a chunk's decays come to, for each event: its sum G as two fp32 numbers (their sum holds 48 bits:
// differences are exact to fp32 whatever pauses lie between), e^G and e^{G_n - G}, in base 2; e^{G_n}.
struct __attribute__((aligned(16))) Decays {
    float hi[kC], lo[kC], from[kC], to[kC];
    float fade;
};

__device__ __forceinline__ float decay_load(const Walk &a, const Part &p, int c, int lane) {
    const int i = c * kC + lane;
    return i < p.len ? a.g[(p.row0 + i) * a.g_row + p.kvh] : 0.f;
}

// 2^x to fp32's precision: what is lost of x in fp32 would be up to 2^-20 of the result.
__device__ __forceinline__ float exp2_of(double x) {
    const float hi = static_cast<float>(x);
    return __builtin_amdgcn_exp2f(hi) * fmaf(static_cast<float>(x - hi), 0.6931471805599453f, 1.f);
}

// By one wavefront, lane = event; adds G_n to *total.
__device__ __forceinline__ void decays(Decays &out, float g, int lane, double *total) {
    g = g > 0.f ? 0.f : g < kLeast ? kLeast : g;  // NaN stays
    const double s = prefix_sum(static_cast<double>(g) * 1.4426950408889634);
    const double n = last_lane(s);
    *total += n;
    const float hi = static_cast<float>(s);
    out.hi[lane] = hi;
    out.lo[lane] = static_cast<float>(s - hi);
    out.from[lane] = exp2_of(s);
    out.to[lane] = exp2_of(n - s);
    if (lane == 0) out.fade = exp2_of(n);
}

// The lane's number, worked out anew: addresses made from it are not kept in registers from one chunk to the next.
__device__ __forceinline__ int fresh(int lane) {
    asm volatile("" : "+v"(lane));
    return lane;
}

// The decays' gradient: none; for each event; for each head (summed over the events).
enum { kNone = 0, kEach = 1, kHead = 2 };

// A barrier for what the wavefronts share in LDS: loads and stores of memory stay under way across it.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The sum over lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float add_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return add_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

template <int LP>
struct Of {
    static constexpr int WAVES = LP / 16, CT = LP / 16, STEPS = LP / 32, TILE = kC * kPitch<LP>;
    typedef floatx4 State[CT];  // tile ct, register r: row 16 ct + 4 quad + r, column 16 w + ln
    typedef floatx4 Out[4];     // rows 16 ib on, register r: column 16 w + 4 quad + r of row 16 ib + ln
};

// Tiles hold each row's columns in the order in which an accumulator holds its rows: of 32, the four from 4 q on
// and those 16 further on are side by side.  So a lane's eight values of an operand are one read, whether the
// other operand comes from a tile or from the accumulators; the order of a product's sum is of no account.
__device__ __forceinline__ constexpr int place_of(int col) { return (col & ~31) + 2 * (col & 12) + (col & 16) / 4 + (col & 3); }

// The 64 rows of a chunk on their way to LDS.  The reads go through a buffer descriptor that ends with the last
// row: past it they give zeros, so that they need no branch (one would wait for reads under way, to carry
// their registers through it), and where nothing is wanted there are no rows.
template <int LP, int THREADS>
struct Loader {
    static constexpr int CH = LP / 8, N = kC * CH / THREADS, R = THREADS / CH;
    u32x4 r[N];
    uint32_t at, step;

    __device__ __forceinline__ Loader(int64_t stride, int d) {
        const int row = threadIdx.x / CH, col = 8 * (threadIdx.x % CH);
        const uint32_t row_bytes = 2 * static_cast<uint32_t>(stride);  // < 2^25
        at = col < d ? row * row_bytes + 2 * col : 0x80000000u;        // columns past the head: past every descriptor
        step = R * row_bytes;
    }
    __device__ __forceinline__ void load(const uint16_t *base, int64_t stride, int d, int rows) {
        rows = min(rows, kC);
        const int64_t bytes = rows > 0 ? 2 * ((rows - 1) * stride + d) : 0;
        const auto desc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(base), 0, static_cast<int>(bytes), 0x00027000);
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(desc, at + i * step, 0, 0));
    }
    // Infinities and NaN become zeros, as 0 times them would reach rows that do not see them: `first` takes the first row of
    // each column that holds one, *any whether there is one.
    __device__ __forceinline__ void tame(int *first, int *any) {
        bool wild = false;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) wild |= (r[i][e] & 0x7f80u) == 0x7f80u || (r[i][e] & 0x7f800000u) == 0x7f800000u;
        if (!wild) return;
        *any = 1;
        const int thread = fresh(threadIdx.x), col = 8 * (thread % CH);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = thread / CH + i * R;
                if ((r[i][e] & 0x7f80u) == 0x7f80u) atomicMin(first + col + 2 * e, row);
                if ((r[i][e] & 0x7f800000u) == 0x7f800000u) atomicMin(first + col + 2 * e + 1, row);
                r[i][e] = only_finite(r[i][e]);
            }
    }
    __device__ __forceinline__ void store(uint16_t *tile) const {
        const int thread = fresh(threadIdx.x);
        uint16_t *const to = tile + thread / CH * kPitch<LP> + place_of(8 * (thread % CH));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            *reinterpret_cast<u32x2 *>(to + i * R * kPitch<LP>) = u32x2{r[i].x, r[i].y};
            *reinterpret_cast<u32x2 *>(to + i * R * kPitch<LP> + 8) = u32x2{r[i].z, r[i].w};
        }
    }
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
__device__ __forceinline__ void state_load(typename Of<LP>::State &S, const float *p, int d, int w, int lane) {
    const int e = 16 * w + (lane & 15);
#pragma unroll
    for (int ct = 0; ct < Of<LP>::CT; ++ct) {
        const int c = 16 * ct + 4 * (lane >> 4);
        S[ct] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (!p || e >= d || c >= d) continue;
        if constexpr (TRANSPOSED) {
            S[ct] = *(const DLRM_GLOBAL floatx4 *)(p + e * d + c);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) S[ct][r] = p[(c + r) * d + e];
        }
    }
}

template <int LP>
__device__ __forceinline__ void state_store(const typename Of<LP>::State &S, float *p, int d, int w, int lane) {
    const int e = 16 * w + (lane & 15);
#pragma unroll
    for (int ct = 0; ct < Of<LP>::CT; ++ct) {
        const int c = 16 * ct + 4 * (lane >> 4);
        if (e >= d || c >= d) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) p[(c + r) * d + e] = S[ct][r];
    }
}

template <int LP>
__device__ __forceinline__ void state_fade(typename Of<LP>::State &S, float f) {
#pragma unroll
    for (int ct = 0; ct < Of<LP>::CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[ct][r] *= f;
}

// Transposed operand of v_mfma_f32_16x16x32_bf16 from a tile: a lane gets column 16 block + ln of the rows
// row0 + 4 quad + {0..3} and those 16 further on.  Within 16 lanes ds_read_b64_tr_b16 takes 4 rows of 16 columns, lane i
// reading 4 columns of row i / 4, and gives lane i column i of the 4 rows.
template <int LP>
__device__ __forceinline__ int columns_base(int lane) {
    return (4 * (lane >> 4) + ((lane & 15) >> 2)) * kPitch<LP> + 8 * (lane & 3);
}
template <int LP>
__device__ __forceinline__ void columns(Frag &f, const uint16_t *at, int row0, int block) {
    typedef __attribute__((address_space(3))) s16x4 *lds_t;
#pragma unroll
    for (int g = 0; g < 2; ++g)
        f.h[g] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(at + (row0 + 16 * g) * kPitch<LP> + 32 * (block / 2) + 4 * (block % 2)));
}

// S <- S + sum_j w_j y_j z_j^T
template <int LP, int UP>
__device__ __forceinline__ void state_grow(typename Of<LP>::State &S, const uint16_t *ys, const uint16_t *zs, const float *weight, int w,
                                           int lane) {
    lane = fresh(lane);
    const uint16_t *const ycol = ys + columns_base<LP>(lane), *const zcol = zs + columns_base<LP>(lane);
    const float *const wj = weight + 4 * (lane >> 4);
#pragma unroll
    for (int s = 0; s < kC / 32; ++s) {
        Frag z, zw[UP];
        columns<LP>(z, zcol, 32 * s, w);
        float x[8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const floatx4 f = *reinterpret_cast<const floatx4 *>(wj + 32 * s + 16 * g);
            x[4 * g] = bf16_lo(z.w[2 * g]) * f[0], x[4 * g + 1] = bf16_hi(z.w[2 * g]) * f[1];
            x[4 * g + 2] = bf16_lo(z.w[2 * g + 1]) * f[2], x[4 * g + 3] = bf16_hi(z.w[2 * g + 1]) * f[3];
        }
        parts_of<UP>(x, zw);
#pragma unroll
        for (int ct = 0; ct < Of<LP>::CT; ++ct) {
            Frag y;
            columns<LP>(y, ycol, 32 * s, ct);
#pragma unroll
            for (int n = 0; n < UP; ++n) S[ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y.b, zw[n].b, S[ct], 0, 0, 0);
        }
    }
}

// o^T = S^T x^T
template <int LP, int PR>
__device__ __forceinline__ void through_state(typename Of<LP>::Out &o, const typename Of<LP>::State &S, const uint16_t *xs, int lane) {
    lane = fresh(lane);
    const uint16_t *const row = xs + (lane & 15) * kPitch<LP> + 8 * (lane >> 4);
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) o[ib] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < Of<LP>::STEPS; ++s) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = S[2 * s + e / 4][e % 4];
        Frag f[PR];
        parts_of<PR>(v, f);
#pragma unroll
        for (int ib = 0; ib < 4; ++ib) {
            Frag x;
            x.q = *reinterpret_cast<const u32x4 *>(row + 16 * ib * kPitch<LP> + 32 * s);
#pragma unroll
            for (int n = 0; n < PR; ++n) o[ib] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[n].b, x.b, o[ib], 0, 0, 0);
        }
    }
}

// Of the 16 tiles of 16 x 16 pairs, the ten that hold some that see each other: tile t has rows 16 jb on of y and 16 ib on
// of x.
constexpr int kTiles = 10;
template <bool REV>
__device__ __forceinline__ void tile_of(int t, int *jb, int *ib) {
    const int a = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3, b = t - a * (a + 1) / 2;
    *ib = REV ? b : a, *jb = REV ? a : b;
}

// Where P holds row i and column j: a row's columns in the order that an operand's lanes take them.
__device__ __forceinline__ int pair_at(int i, int j) { return i * kPP + (j & 32) + 2 * (j & 12) + (j & 16) / 4 + (j & 3); }

// The tiles beside the diagonal that a product of 32 columns takes along are zeros, once and for all.
template <bool REV>
__device__ __forceinline__ void pair_zeros(uint16_t *P, int t) {
    if (t >= 128) return;
    const int i = (t & 64 ? 32 : 0) + (REV ? 16 : 0) + (t & 15), j = (t & 64 ? 32 : 0) + (REV ? 0 : 16) + (t & 48) / 4;
    *reinterpret_cast<u32x2 *>(P + pair_at(i, j)) = u32x2{0, 0};
}

// P^T = <y_j, x_i> e^{..}, rounded to bf16, one tile, to LDS.  With a second pair of rows: the same of it to P2 (BOTH);
// GRAD: sums over j of both products times e^{..}, for each i (kept unrounded: the decays' gradient is fp32), for each head
// times the events between the two.
template <int LP, bool REV, bool BOTH, int GRAD>
__device__ __forceinline__ float pair_tile(uint16_t *P, uint16_t *P2, const Decays &dec, const uint16_t *xs, const uint16_t *ys,
                                           const uint16_t *x2s, const uint16_t *y2s, int t, int lane) {
    lane = fresh(lane);
    int jb, ib;
    tile_of<REV>(t, &jb, &ib);
    const int ln = lane & 15, quad = lane >> 4;
    const int xat = (16 * ib + ln) * kPitch<LP> + 8 * quad, yat = (16 * jb + ln) * kPitch<LP> + 8 * quad;
    floatx4 s = {0.f, 0.f, 0.f, 0.f}, m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < Of<LP>::STEPS; ++i) {
        Frag x, y;
        x.q = *reinterpret_cast<const u32x4 *>(xs + xat + 32 * i);
        y.q = *reinterpret_cast<const u32x4 *>(ys + yat + 32 * i);
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y.b, x.b, s, 0, 0, 0);
        if constexpr (BOTH || GRAD != kNone) {
            Frag u, v;
            u.q = *reinterpret_cast<const u32x4 *>(x2s + xat + 32 * i);
            v.q = *reinterpret_cast<const u32x4 *>(y2s + yat + 32 * i);
            m = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v.b, u.b, m, 0, 0, 0);
        }
    }
    const int i = 16 * ib + ln, j0 = 16 * jb + 4 * quad;
    const float hi = dec.hi[i], lo = dec.lo[i];
    const floatx4 hj = *reinterpret_cast<const floatx4 *>(dec.hi + j0), lj = *reinterpret_cast<const floatx4 *>(dec.lo + j0);
    float p[4], p2[4], sum = 0.f;
    const auto pair = [&](int r, bool sees) {
        const float diff = REV ? (hj[r] - hi) + (lj[r] - lo) : (hi - hj[r]) + (lo - lj[r]);
        const float e = __builtin_amdgcn_exp2f(diff);
        p[r] = sees ? s[r] * e : 0.f;
        if constexpr (BOTH) p2[r] = sees ? m[r] * e : 0.f;
        if constexpr (GRAD == kEach) sum = fmaf(p[r], m[r], sum);
        if constexpr (GRAD == kHead) sum = fmaf(p[r] * static_cast<float>(REV ? j0 + r - i : i - j0 - r), m[r], sum);
    };
    if (ib == jb) {
#pragma unroll
        for (int r = 0; r < 4; ++r) pair(r, REV ? j0 + r >= i : j0 + r <= i);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) pair(r, true);
    }
    const int at = pair_at(i, j0);
    *reinterpret_cast<u32x2 *>(P + at) = u32x2{pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3])};
    if constexpr (BOTH) *reinterpret_cast<u32x2 *>(P2 + at) = u32x2{pack_bf16(p2[0], p2[1]), pack_bf16(p2[2], p2[3])};
    return GRAD != kNone ? add_quarters(sum) : 0.f;
}

// o^T += z^T P^T
template <int LP, bool REV>
__device__ __forceinline__ void through_pairs(typename Of<LP>::Out &o, const uint16_t *P, const uint16_t *zs, int w, int lane) {
    lane = fresh(lane);
    const uint16_t *const zcol = zs + columns_base<LP>(lane);
    const uint16_t *const row = P + (lane & 15) * kPP + 8 * (lane >> 4);
#pragma unroll
    for (int s = 0; s < kC / 32; ++s) {
        Frag z;
        columns<LP>(z, zcol, 32 * s, w);
#pragma unroll
        for (int ib = 0; ib < 4; ++ib) {
            if (REV ? ib / 2 > s : ib / 2 < s) continue;  // none of its pairs see each other
            Frag p;
            p.q = *reinterpret_cast<const u32x4 *>(row + 16 * ib * kPP + 32 * s);
            o[ib] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z.b, p.b, o[ib], 0, 0, 0);
        }
    }
}

// NaN for what z held infinities or NaN for (Loader::tame): the rows from the first such one on, and the state.
__device__ __forceinline__ void out_wild(floatx4 (&o)[4], const int *first, int w, int lane) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int from = first[16 * w + 4 * (lane >> 4) + r];
#pragma unroll
        for (int ib = 0; ib < 4; ++ib)
            if (16 * ib + (lane & 15) >= from) o[ib][r] = __builtin_nanf("");
    }
}
template <int LP>
__device__ __forceinline__ void state_wild(typename Of<LP>::State &S, const int *first, int w, int lane) {
    if (first[16 * w + (lane & 15)] < kC) state_fade<LP>(S, __builtin_nanf(""));
}

// o times f of each row; MORE: *sums of o's columns times those of the row of t, for rows 16 ib + ln.
template <int LP, bool MORE>
__device__ __forceinline__ void weigh(typename Of<LP>::Out &o, const float *f, const uint16_t *ts, float *sums, int w, int lane) {
    lane = fresh(lane);
    const int ln = lane & 15, quad = lane >> 4;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib) {
        const int row = 16 * ib + ln;
        const float x = f[row];
#pragma unroll
        for (int r = 0; r < 4; ++r) o[ib][r] *= x;
        if constexpr (MORE) {
            const u32x2 t = *reinterpret_cast<const u32x2 *>(ts + row * kPitch<LP> + place_of(16 * w) + 8 * quad);
            const float sum = add_quarters(o[ib][0] * bf16_lo(t.x) + o[ib][1] * bf16_hi(t.x) +
                                           (o[ib][2] * bf16_lo(t.y) + o[ib][3] * bf16_hi(t.y)));
            if (quad == 0) sums[row] = sum;
        }
    }
}

// Rows of one chunk's outputs, a wavefront's columns, by way of that part of a tile that nobody reads any more
// (from the accumulators a store would write 8 bytes of each of 16 rows).
template <int LP>
__device__ __forceinline__ void out_rows(const typename Of<LP>::Out &o, uint16_t *tile, uint16_t *out, int64_t stride, int rows, int d,
                                         float scale, int w, int lane) {
    lane = fresh(lane);
    const int ln = lane & 15, quad = lane >> 4;
    uint16_t *const part = tile + 16 * w;
#pragma unroll
    for (int ib = 0; ib < 4; ++ib)
        *reinterpret_cast<u32x2 *>(part + (16 * ib + ln) * kPitch<LP> + 4 * quad) =
            u32x2{pack_bf16(o[ib][0] * scale, o[ib][1] * scale), pack_bf16(o[ib][2] * scale, o[ib][3] * scale)};
    wave_lds_sync();
    const int col = 8 * (lane & 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 32 * i + (lane >> 1);
        if (row < rows && 16 * w + col < d)
            *(DLRM_GLOBAL u32x4 *)(out + row * stride + 16 * w + col) = *reinterpret_cast<const u32x4 *>(part + row * kPitch<LP> + col);
    }
}

// ---------------------------------------------------------------- host

// Checks the description and fills what all walks share.
int check(const dlrm_seq_decay *a, bool offsets, Walk *out);

inline uint32_t workgroups_of(const Walk &a) { return (a.slots + kNumXcd - 1) / kNumXcd * kNumXcd * a.Hkv * a.splits; }

// How sequences are cut: chunks of a run (0: not), and slots; `back`: for the backward.
struct Cut {
    int32_t run;
    int64_t slots;
    bool order;  // sequences go by their length
};
Cut cut_of(const Walk &a, int64_t max_len, bool back);

constexpr int padded(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }
constexpr size_t whole(size_t bytes) { return (bytes + 255) / 256 * 256; }

// Bytes of one direction's states and fades of runs, and of the order.
size_t states_bytes(const Walk &a, const Cut &c);
size_t order_bytes(const Walk &a, const Cut &c);

// The order of the sequences, into `order`.
int order_by_length(const Walk &a, int32_t *order, hipStream_t stream);

// The states at the start of every run after a sequence's first one: of `f` (its y and z) forward and, unless it is NULL,
// of `r` reversed, into the `start` of each.
int run_states(const Walk &f, const Walk *r, int up, hipStream_t stream);

// Workgroups that share a group's query heads in the forward walk.
int splits_of(const Walk &a, bool back);

// The forward walk; `up`, `grad`: the kernel's.
int walk(const Walk &a, int up, int grad, hipStream_t stream);

}  // namespace decay
}  // namespace seq
}  // namespace dlrm
