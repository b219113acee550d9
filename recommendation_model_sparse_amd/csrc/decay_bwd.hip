// Linear attention with a decay, backward (dlrm_seq_decay.h): dq by the forward walk on (do, v, k), dk and dv by
// a walk in reverse time, dg from both.
#include "decay.h"

namespace dlrm {
namespace seq {
namespace decay {
namespace {

// dk and dv in one walk from a sequence's end: two teams of wavefronts over the same tiles, the first for dv
// (x = k, y = q, z = do), the second for dk (x = v, y = do, z = q); the state of the second is the first's, transposed,
// and laid out as that of the walk for dq.  a.x, a.y, a.z, a.t: k, q, do, v; a.out: dv, a.out2: dk; a.start: the
// first team's states.
//
// GRAD: dg.  With x_i and y_j what <q_i, dq_i> and <k_j, dk_j> have by way of the states (of pairs in different chunks), r_i and
// c_j what they have within the chunk, and Z = <S, R> all pairs across the chunk's end at once, S the forward state
// there (dq's), R the one of this walk:
//
//     dg_t = Z + sum_{i>=t} (x_i - y_i) + sum_{i>=t} (r_i - c_i)
//
// and Z at the chunk's beginning is the first two parts for its first event (the third is zero there, but for its
// rounding, which is left out).  Such sums cancel, and rounding would add up over a long sequence: at the marks Z is taken
// from the states themselves.  Over all events of a head: n Z + sum (i + 1) (x_i - y_i) + the pairs times the events between
// them, i and n within the chunk.
//
// Both teams share the tiles of k, v, q and do (one read of each from memory), the decays and the ten tiles of pairs: each
// <k, q> and <v, do> is worked out once.  LDS holds two workgroups a CU of heads of 64, one of 128, and registers four
// wavefronts a SIMD.  UP, PR: as in the forward walk.  Heads of 128 spill 4 vector registers with dg, 20 bytes of scratch a lane, and
// 288 without, 388 bytes: 65 us where 55 with dg, for the 4 sequences below (the whole backward 117 and 124).
// Measured, by the profiler: 1024 sequences of 16 to 512, 2 heads of 64, 94 us: VALU 54 %, LDS 37 %, MFMA 18 %, 2.4 TB/s; 4 of 2000 to 4096, 8
// heads of 128 over 2 in runs of two chunks, 56 us: 28, 23, 18 %, one workgroup a CU.
template <int LP, int UP, int PR, int GRAD>
__global__ __launch_bounds__(Of<LP>::WAVES * 128, LP == 32 ? 3 : 4) void k_decay_back(const Walk a) {
    using O = Of<LP>;
    constexpr bool MORE = GRAD != kNone;
    constexpr int TEAM = 64 * O::WAVES, THREADS = 2 * TEAM;
    __shared__ __attribute__((aligned(16))) uint16_t Ks[O::TILE], Vs[O::TILE], Qs[O::TILE], Ds[O::TILE], Ps[2][kC * kPP];
    __shared__ __attribute__((aligned(16))) Decays decs[2];
    __shared__ float by_wave[MORE ? O::WAVES : 1][kC], by_tile[MORE ? kTiles : 1][16];
    __shared__ double across[MORE ? O::WAVES : 1];

    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, quad = lane >> 4;
    const Part p = part_of(a);
    if (!p.any) {
        if (GRAD == kHead && p.slot < a.slots && tid == 0) a.sums[static_cast<int64_t>(p.kvh) * a.slots + p.slot] = 0.0;
        return;
    }
    const int team = static_cast<int>(wave_id()) / O::WAVES, w = static_cast<int>(wave_id()) % O::WAVES;
    const int h0 = p.kvh * a.group;
    const uint16_t *kb = a.x.p + p.row0 * a.x.row + p.kvh * a.x.head;
    const uint16_t *vb = a.t.p + p.row0 * a.t.row + p.kvh * a.t.head;
    const uint16_t *qb = a.y.p + p.row0 * a.y.row + h0 * a.y.head;
    const uint16_t *db = a.z.p + p.row0 * a.z.row + h0 * a.z.head;
    uint16_t *const xt = team ? Vs : Ks;
    const uint16_t *const yt = team ? Ds : Qs, *const zt = team ? Qs : Ds;
    uint16_t *const P = Ps[team];

    Loader<LP, THREADS> ks(a.x.row, a.d), vs(a.t.row, a.d), qs(a.y.row, a.d), ds(a.z.row, a.d);
    const auto load = [&](int c, int h) {  // of k and v with the first head
        const int rows = c >= p.c0 ? p.len - c * kC : 0;
        const int64_t row = static_cast<int64_t>(c) * kC;
        ks.load(kb + row * a.x.row, a.x.row, a.d, h == 0 ? rows : 0);
        vs.load(vb + row * a.t.row, a.t.row, a.d, h == 0 ? rows : 0);
        qs.load(qb + row * a.y.row + h * a.y.head, a.y.row, a.d, rows);
        ds.load(db + row * a.z.row + h * a.z.head, a.z.row, a.d, rows);
    };
    const bool clock = team == 0 && w == O::WAVES - 1;
    float g = 0.f;
    double total = 0.0, carry = 0.0, all = 0.0;
    if (p.c0 < p.c1) {
        if (clock) g = decay_load(a, p, p.c1 - 1, lane);
    }
    load(p.c1 - 1, 0);
    typename O::State S;
    const float *start = p.c1 < p.chunks ? a.start + (p.slot * static_cast<int64_t>(a.Hkv) + p.kvh) * a.d * a.d : nullptr;
    if (team) state_load<LP, true>(S, start, a.d, w, lane);
    else state_load<LP, false>(S, start, a.d, w, lane);
    pair_zeros<true>(P, tid - team * TEAM);
    if (clock && p.c0 < p.c1) {
        decays(decs[(p.c1 - 1) & 1], g, lane, &total);
        if (p.c1 - 2 >= p.c0) g = decay_load(a, p, p.c1 - 2, lane);
    }
    // The pairs across the beginning of chunk c, in the state that the chunks from it on have left.
    const auto begin_anew = [&](int c) {
        if (team) {
            const float *at = a.marks + mark_at(a, p, c) * (LP * LP) + 4 * (tid - TEAM);
            double sum = 0.0;
#pragma unroll
            for (int ct = 0; ct < O::CT; ++ct) {
                const floatx4 f = *(const DLRM_GLOBAL floatx4 *)(at + ct * 4 * TEAM);
#pragma unroll
                for (int r = 0; r < 4; ++r) sum += static_cast<double>(f[r]) * S[ct][r];
            }
#pragma unroll
            for (int i = 1; i < 64; i <<= 1) sum += __shfl_xor(sum, i);
            if (lane == 0) across[w] = sum;
        }
        lds_barrier();
        carry = 0.0;
        for (int v = 0; v < O::WAVES; ++v) carry += across[v];
        carry *= a.scale;
    };
    if (MORE && p.c0 < p.c1 && p.c1 < p.chunks) begin_anew(p.c1);

    for (int c = p.c1 - 1; c >= p.c0; --c) {
        const Decays &dec = decs[c & 1];
        const int rows = min(kC, p.len - c * kC);
        typename O::Out o;
        float term = 0.f, pairs = 0.f, plus = 0.f, plus_pairs = 0.f, here = 0.f;
        for (int h = 0; h < a.group; ++h) {
            lds_barrier();  // the tiles before have been read
            if (h == 0) ks.store(Ks), vs.store(Vs);
            qs.store(Qs), ds.store(Ds);
            lds_barrier();
            load(h + 1 < a.group ? c : c - 1, h + 1 < a.group ? h + 1 : 0);
            if (clock && h == 0 && c > p.c0) {
                decays(decs[~c & 1], g, lane, &total);
                if (c - 2 >= p.c0) g = decay_load(a, p, c - 2, lane);
            }
            if (MORE && tid < 64 && h == 0 && lane < rows) {
                const int64_t row = p.row0 + c * kC + lane;
                here = a.g[row * a.g_row + p.kvh];
                for (int s = 0; s < a.parts; ++s) {
                    const int64_t at = (s * static_cast<int64_t>(a.Hkv) + p.kvh) * a.N + row;
                    plus += a.terms[at];
                    if constexpr (GRAD == kEach) plus_pairs += a.pairs[at];
                }
            }
            // both teams' pairs, tile by tile: they have their decays in common, and dg takes the product of both
#pragma unroll
            for (int n = 0; n < (kTiles + 2 * O::WAVES - 1) / (2 * O::WAVES); ++n) {
                const int t = static_cast<int>(wave_id()) + n * 2 * O::WAVES;
                if (t >= kTiles) break;
                const float sum = pair_tile<LP, true, true, GRAD>(Ps[0], Ps[1], dec, Ks, Qs, Vs, Ds, t, lane);
                if constexpr (MORE) {
                    if (quad == 0) by_tile[t][ln] = sum;
                }
            }
            if (h == 0) {
                through_state<LP, PR>(o, S, xt, lane);
                if (MORE && team == 1) weigh<LP, MORE>(o, dec.to, Ks, by_wave[MORE ? w : 0], w, lane);
                else weigh<LP, false>(o, dec.to, nullptr, nullptr, w, lane);
                state_fade<LP>(S, dec.fade);
            }
            lds_barrier();
            through_pairs<LP, true>(o, P, zt, w, lane);
            state_grow<LP, UP>(S, yt, zt, dec.from, w, lane);
            if (MORE && tid < 64) {
                const int ib = lane / 16;  // tile (a, b) is number a (a + 1) / 2 + b and has the rows 16 b on
                for (int t = ib; t < 4; ++t) pairs += by_tile[t * (t + 1) / 2 + ib][ln];
                if (h == 0) {
#pragma unroll
                    for (int v = 0; v < O::WAVES; ++v) term += by_wave[v][lane];
                }
            }
        }
        out_rows<LP>(o, xt, (team ? a.out2 : a.out) + ((p.row0 + c * kC) * a.Hkv + p.kvh) * a.d, static_cast<int64_t>(a.Hkv) * a.d, rows, a.d,
                     a.scale, w, lane);
        if constexpr (MORE) {
            if (tid < 64) {
                const bool in = lane < rows;
                const double x = in ? static_cast<double>(plus) - static_cast<double>(term * a.scale) : 0.0;
                if constexpr (GRAD == kEach) {
                    const double y = in ? static_cast<double>(plus_pairs) - static_cast<double>(pairs * a.scale) : 0.0;
                    const double upto = prefix_sum(x + y), n = last_lane(upto);
                    const double after = here > 0.f ? 0.0 : carry + (n - upto + x + y);  // from this event on
                    if (in) a.dg[(p.row0 + c * kC + lane) * a.Hkv + p.kvh] = static_cast<float>(after);
                } else if (in && !(here > 0.f)) {
                    all += carry + (lane + 1) * x + static_cast<double>(pairs * a.scale);
                }
                carry += last_lane(prefix_sum(x));
            }
            if (c > p.c0 && c % a.mark == 0) begin_anew(c);
        }
    }
    if (GRAD == kHead && tid < 64) {
        all = last_lane(prefix_sum(all));
        if (lane == 0) a.sums[static_cast<int64_t>(p.kvh) * a.slots + (a.run ? p.slot : p.b)] = all;  // not by their order, which is left to chance
    }
}

// dg of one decay a head: over the slots, in a fixed order.
__global__ __launch_bounds__(256) void k_decay_dg_join(const double *sums, uint32_t slots, float *dg) {
    __shared__ double part[4];
    const int lane = threadIdx.x & 63, w = static_cast<int>(wave_id());
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < slots; i += 256) s += sums[static_cast<int64_t>(blockIdx.x) * slots + i];
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) s += __shfl_xor(s, i);
    if (lane == 0) part[w] = s;
    __syncthreads();
    if (threadIdx.x == 0) dg[blockIdx.x] = static_cast<float>(part[0] + part[1] + part[2] + part[3]);
}

template <int LP>
int back(const Walk &a, int grad, hipStream_t stream) {
    const dim3 grid(workgroups_of(a)), block(Of<LP>::WAVES * 128);
    if (grad == kEach) DLRM_LAUNCH("seq_decay_dkv", (k_decay_back<LP, 3, 3, kEach>), grid, block, 0, stream, a);
    else if (grad == kHead) DLRM_LAUNCH("seq_decay_dkv", (k_decay_back<LP, 3, 3, kHead>), grid, block, 0, stream, a);
    else DLRM_LAUNCH("seq_decay_dkv", (k_decay_back<LP, 2, 1, kNone>), grid, block, 0, stream, a);
    return launch_status();
}

// Marks are eight chunks apart, or two where dg is summed over the events, which leaves an error of Z in every event of
// a chunk; or a run's length, or one: at every run's start there is one.  (Two decays over 29000 events: an error of 7e-5 of the sum
// without the marks between, as the events' own errors are 6e-7.)
int mark_of(const Cut &c, bool by_head) { return by_head ? 2 - c.run % 2 : c.run && c.run < 8 ? c.run : 8; }

// Bytes: the runs' states, forward and reversed, or the order; for dg, the terms from dq, the states at the marks, the
// slots' sums.
struct Room {
    size_t states, order, terms, marks, sums;
};
Room room_of(Walk a, const Cut &c) {
    a.slots = static_cast<uint32_t>(c.slots);
    const size_t lp = padded(a.d);
    return Room{states_bytes(a, c), order_bytes(a, c), whole(8 * static_cast<size_t>(a.N) * a.Hkv * splits_of(a, true)),
                4 * lp * lp * a.Hkv * static_cast<size_t>(a.N / (kC * mark_of(c, a.g_row == 0))),
                whole(8 * static_cast<size_t>(c.slots) * a.Hkv)};
}

}  // namespace
}  // namespace decay
}  // namespace seq
}  // namespace dlrm

extern "C" size_t dlrm_seq_decay_bwd_workspace_size(const dlrm_seq_decay *desc) {
    using namespace dlrm::seq::decay;
    Walk a;
    if (check(desc, true, &a) != DLRM_OK) return 0;
    const Room r = room_of(a, cut_of(a, desc->max_len, true));
    return 256 + 2 * r.states + r.order + r.terms + r.marks + r.sums;
}

extern "C" int dlrm_seq_decay_bwd(const dlrm_seq_decay *desc, const uint16_t *dout, uint16_t *dq, uint16_t *dk, uint16_t *dv, float *dg,
                                  void *workspace, size_t workspace_bytes, dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq::decay;
    Walk a;
    int rc = check(desc, true, &a);
    if (rc != DLRM_OK) return rc;
    if (a.N > 0 && (!dout || !dq || !dk || !dv)) return DLRM_ERR_INVALID_ARG;
    if (!aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(dg, 4)) return DLRM_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < dlrm_seq_decay_bwd_workspace_size(desc)) return DLRM_ERR_WORKSPACE;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    const bool by_head = dg && a.g_row == 0, any = a.N > 0 && a.B > 0;
    const int grad = !dg ? kNone : by_head ? kHead : kEach, up = dg ? 3 : 2;
    const Cut c = cut_of(a, desc->max_len, true);
    const Room room = room_of(a, c);
    char *ws = static_cast<char *>(workspace);
    const auto take = [&](size_t bytes) {
        char *p = ws;
        ws += bytes;
        return p;
    };
    float *forward = reinterpret_cast<float *>(take(room.states)), *reversed = reinterpret_cast<float *>(take(room.states));
    int32_t *order = reinterpret_cast<int32_t *>(take(room.order));
    a.terms = reinterpret_cast<float *>(take(room.terms)), a.marks = reinterpret_cast<float *>(take(room.marks));
    double *sums = reinterpret_cast<double *>(take(room.sums));
    a.run = c.run, a.slots = static_cast<uint32_t>(c.slots), a.mark = mark_of(c, by_head);
    const int splits = splits_of(a, true);
    a.pairs = a.terms + a.N * a.Hkv * splits;
    if (any) {
        const Heads q = a.x, k = a.y, v = a.z, d = {dout, static_cast<int64_t>(a.Hq) * a.d, a.d};
        Walk r = a;
        a.x = d, a.y = v, a.z = k, a.t = q, a.out = dq;
        r.x = k, r.y = q, r.z = d, r.t = v, r.out = dv, r.out2 = dk;
        r.parts = splits, r.dg = dg, r.sums = sums;
        if (c.run) {
            const int64_t states = c.slots * a.Hkv * a.d * a.d;
            a.start = forward, a.fade = forward + states;
            r.start = reversed, r.fade = reversed + states;
            rc = run_states(a, &r, up, stream);
        } else if (c.order) {
            rc = order_by_length(a, order, stream);
            a.order = r.order = order;
        }
        if (rc != DLRM_OK) return rc;
        a.splits = splits;
        rc = walk(a, up, grad, stream);
        if (rc != DLRM_OK) return rc;
        rc = a.d <= 32 ? back<32>(r, grad, stream) : a.d <= 64 ? back<64>(r, grad, stream) : back<128>(r, grad, stream);
        if (rc != DLRM_OK) return rc;
    }
    if (by_head)
        DLRM_LAUNCH("seq_decay_dg_join", k_decay_dg_join, dim3(a.Hkv), dim3(256), 0, stream, static_cast<const double *>(sums),
                    any ? a.slots : 0u, dg);
    return launch_status();
}
