// Linear attention with a decay, forward (dlrm_seq_decay.h), and what its backward shares: the forward walk
// (outputs, or dq), the states at the start of runs, the checks.
#include <algorithm>

#include "decay.h"

namespace dlrm {
namespace seq {
namespace decay {

int check(const dlrm_seq_decay *a, bool offsets, Walk *out) {
    if (!a) return DLRM_ERR_INVALID_ARG;
    if (a->B < 0 || a->N < 0 || a->Hq < 1 || a->Hkv < 1 || a->Hq % a->Hkv != 0 || a->d < 1) return DLRM_ERR_INVALID_ARG;
    if (a->index_type != DLRM_INDEX_I64 && a->index_type != DLRM_INDEX_I32) return DLRM_ERR_INVALID_ARG;
    if (!(a->scale == a->scale) || a->max_len < 0 || (a->g_row != 0 && a->g_row < a->Hkv)) return DLRM_ERR_INVALID_ARG;
    if (a->d % 8 != 0 || a->d > 128 || a->Hq > 4096 || a->B >= (1 << 24) || a->N >= (int64_t(1) << 31)) return DLRM_ERR_UNSUPPORTED;
    if (offsets) {
        const uintptr_t ib = a->index_type == DLRM_INDEX_I32 ? 4 : 8;
        if (a->B > 0 && (!a->offsets || !aligned(a->offsets, ib))) return DLRM_ERR_INVALID_ARG;
        // a launch holds fewer than 2^32 work-items
        if ((slot_count(a->N, a->B, kC) + kNumXcd) * a->Hkv >= (int64_t(1) << (a->d <= 64 ? 23 : 22))) return DLRM_ERR_UNSUPPORTED;
    }
    if (a->N > 0 && (!a->q || !a->k || !a->v || !a->g)) return DLRM_ERR_INVALID_ARG;
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->g, 4)) return DLRM_ERR_INVALID_ARG;
    const int64_t strides[6] = {a->q_row, a->q_head, a->k_row, a->k_head, a->v_row, a->v_head};
    for (int64_t s : strides)
        if (s % 8 != 0 || s < a->d) return DLRM_ERR_INVALID_ARG;
    for (int i = 0; i < 6; i += 2)
        if (strides[i] >= (1 << 24)) return DLRM_ERR_UNSUPPORTED;  // a tile's rows are 32-bit offsets apart
    if (a->g_row >= (1 << 24)) return DLRM_ERR_UNSUPPORTED;
    *out = Walk{};
    out->x = Heads{a->q, a->q_row, a->q_head};
    out->y = Heads{a->k, a->k_row, a->k_head};
    out->z = Heads{a->v, a->v_row, a->v_head};
    out->g = a->g, out->g_row = a->g_row;
    out->off = a->offsets, out->idx32 = a->index_type == DLRM_INDEX_I32;
    out->N = a->N, out->B = static_cast<int32_t>(a->B);
    out->Hq = a->Hq, out->Hkv = a->Hkv, out->group = a->Hq / a->Hkv, out->d = a->d;
    out->scale = a->scale, out->splits = 1;
    return DLRM_OK;
}

// Most sequences that one workgroup puts in order; chunks of the longest run, whose rows are an int's.
constexpr int kOrdered = 16384, kMostChunks = 1 << 20;
constexpr int kCUs = 256;

// Workgroups that are resident at once, as their LDS leaves room for them: of the forward walk, of k_decay_back.
static int places_of(int32_t d, bool back) {
    const int lp = padded(d);
    return kCUs * (back ? (lp == 32 ? 3 : lp == 64 ? 2 : 1) : (lp == 32 ? 5 : lp == 64 ? 4 : 2));
}

// Heads of a group are split where there are so few workgroups that two times as many would still have places (4 long
// histories, 8 heads of 128 over 2: without 47 us, split until all places are taken 50, like this 43; one of 400, 16 heads over
// 2: 51, 21, 21).
static int splits_for(int64_t workgroups, int group, int places) {
    int n = 1;
    while (n < group && workgroups * n < places / 2) {
        do ++n;
        while (group % n != 0);
    }
    return n;
}

// A sequence and key head a workgroup is enough where there are many; where few are long, they are cut into
// runs, whose states at the start are made first from y and z alone.  What takes least is worked out, in chunks of one head:
// a workgroup begins in the time of 2 and takes its heads' chunks and, cut, one more for the states; workgroups past
// the places wait for others, and the last of them ends three quarters of its own time after the mean; joining the states
// takes 1 for each 16 runs of the longest sequence, and the two launches 2.  Of the runs of 1 to 8 and 16 chunks and none, on
// 17 shapes forward and backward (1 to 1024 sequences of 1 to 8192, heads of 32, 64, 128, groups of 1 to 16), this choice
// was 0.4 % slower than the best in the mean, 10 % at worst.
// The states of the runs, one a sequence among them, are held to what the rows of q, k, v and o take, or to what the 256 MB behind
// the L2s hold: with an unknown longest history the time alone would cut any batch, as one sequence might be all of it (20000
// histories of 60 events, 4 heads of 128, are left whole, where runs would take 5.4 GB of states beside 4.9 GB of rows; of 1 to 120,
// 0.49 million events: 2693 -> 1153 us, the backward 9980 -> 6584).
Cut cut_of(const Walk &a, int64_t max_len, bool back) {
    const int64_t longest = (std::min(max_len, a.N) + kC - 1) / kC;
    const int places = places_of(a.d, back);
    const double total = static_cast<double>(slot_count(a.N, a.B, kC) * a.Hkv);
    const auto time_of = [&](int64_t run) {
        const int64_t groups = (run ? slot_count(a.N, a.B, kC * static_cast<int>(run)) : a.B) * a.Hkv;
        const double heads = back ? a.group : a.group / splits_for(groups, a.group, places), each = heads + (run ? 1 : 0);
        const double own = (run ? run : longest) * each;
        const double shared = (total * each + 2.0 * groups) / places;
        if (!run) return std::max(own + 2, shared);
        return (groups <= places ? own + 2 : shared + 0.75 * own) + 2 + (longest / run + 15) / 16;
    };
    const int64_t room = std::max(int64_t(1) << 28, 4 * a.N * a.d * (a.Hq + a.Hkv));
    const auto fits = [&](int64_t run) { return slot_count(a.N, a.B, kC * static_cast<int>(run)) * a.Hkv <= room / (4 * a.d * a.d); };
    Cut c = {};
    double least = time_of(0);
    const bool many = a.B * static_cast<int64_t>(a.Hkv) * 64 >= (int64_t(1) << 24);  // more than a launch of k_decay_join holds
    // (from 8 on, multiples of 8: the marks are that far apart)
    for (int64_t run = 1; run < longest && run <= kMostChunks && !many; run += run < 8 ? 1 : run) {
        const double t = time_of(run);
        if (t < least && fits(run)) least = t, c.run = static_cast<int32_t>(run);
    }
    c.slots = c.run ? slot_count(a.N, a.B, kC * c.run) : a.B;
    // the longest first: with 1024 sequences of 16 to 512, 2 heads of 64, 42 us instead of 56, the backward 143 instead of 202
    c.order = !c.run && longest > 1 && a.B <= kOrdered && static_cast<int64_t>(a.B) * a.Hkv > places / 2;
    return c;
}

size_t states_bytes(const Walk &a, const Cut &c) {
    return c.run ? whole(4 * static_cast<size_t>(c.slots) * a.Hkv * (static_cast<size_t>(a.d) * a.d + 1)) : 0;
}
size_t order_bytes(const Walk &a, const Cut &c) { return c.order ? whole(4 * static_cast<size_t>(a.B)) : 0; }

int splits_of(const Walk &a, bool back) {
    return splits_for(static_cast<int64_t>(a.slots) * a.Hkv, a.group, places_of(a.d, back));
}

namespace {

// The forward walk: o, or dq with what dg takes from it.  UP, PR: bf16 parts of w_j z_j as the state grows, of the state as
// the outputs take it.  The state: two parts (2^-16) where only outputs in bf16 come of it, three (2^-24) where it or dg is an output;
// outputs take it rounded (PR 1), but dg's terms are fp32's.  (Two parts with dg: 4 % faster, and dg 3e-6 off instead of 4e-7.)
// A head is three steps between barriers: tiles to LDS; pairs, and what comes through the state, with the next rows under
// way; what comes through the pairs.  The registers leave room for as many workgroups as LDS does: heads of 64 four a CU,
// three with dg.  (Heads of 128 without dg: five vector registers spilled, 24 bytes of scratch a lane.)
// Measured, by the profiler: heads of 64, 1024 sequences of 16 to 512, 2 heads: o 38 us, 3.8 TB/s; dq 61.  Heads of 128, 64 sequences of 1 to 1500
// with states, 8 heads over 2: 31 us, and 22 for the states at the runs' starts.
template <int LP, int UP, int PR, int GRAD>
__global__ __launch_bounds__(Of<LP>::WAVES * 64, LP == 128 ? (GRAD ? 2 : 4) : LP == 64 ? (GRAD ? 3 : 4) : GRAD ? 2 : 3) void k_decay_walk(const Walk a) {
    constexpr bool MORE = GRAD != kNone;
    using O = Of<LP>;
    constexpr int THREADS = 64 * O::WAVES;
    __shared__ __attribute__((aligned(16))) uint16_t Xs[O::TILE], Ys[O::TILE], Zs[O::TILE], P[kC * kPP];
    __shared__ __attribute__((aligned(16))) Decays decs[2];
    __shared__ __attribute__((aligned(16))) uint16_t Ts[MORE ? O::TILE : 8];
    __shared__ float by_wave[MORE ? O::WAVES : 1][kC], by_tile[GRAD == kEach ? kTiles : 1][16];
    __shared__ int wild[2], first_wild[2][LP];  // infinities and NaN in z (Loader::tame), in even and odd chunks

    const Part p = part_of(a);
    if (!p.any) return;
    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, quad = lane >> 4;
    const int w = static_cast<int>(wave_id());
    const int heads = a.group / a.splits, h0 = p.kvh * a.group + p.split * heads;
    const uint16_t *xb = a.x.p + p.row0 * a.x.row + h0 * a.x.head;
    const uint16_t *yb = a.y.p + p.row0 * a.y.row + p.kvh * a.y.head;
    const uint16_t *zb = a.z.p + p.row0 * a.z.row + p.kvh * a.z.head;
    const uint16_t *tb = MORE ? a.t.p + p.row0 * a.t.row + h0 * a.t.head : nullptr;

    Loader<LP, THREADS> xs(a.x.row, a.d), ys(a.y.row, a.d), zs(a.z.row, a.d), ts(MORE ? a.t.row : 0, a.d);
    const auto load = [&](int c, int h) {  // of y and z with the first head
        const int rows = c < p.c1 ? p.len - c * kC : 0;
        const int64_t row = static_cast<int64_t>(c) * kC;
        ys.load(yb + row * a.y.row, a.y.row, a.d, h == 0 ? rows : 0);
        zs.load(zb + row * a.z.row, a.z.row, a.d, h == 0 ? rows : 0);
        xs.load(xb + row * a.x.row + h * a.x.head, a.x.row, a.d, rows);
        if constexpr (MORE) ts.load(tb + row * a.t.row + h * a.t.head, a.t.row, a.d, rows);
    };
    const bool clock = w == O::WAVES - 1;  // the wavefront that works out the next chunk's decays: it has the fewest tiles
    float g = 0.f;
    double total = 0.0;
    if (p.c0 < p.c1) {
        if (clock) g = decay_load(a, p, p.c0, lane);
    }
    load(p.c0, 0);
    typename O::State S;
    const int64_t dd = static_cast<int64_t>(a.d) * a.d;
    const float *start = a.first ? a.first + (static_cast<int64_t>(p.b) * a.Hkv + p.kvh) * dd : nullptr;
    if (p.c0 > 0 || a.all_start) start = a.start + (p.slot * static_cast<int64_t>(a.Hkv) + p.kvh) * dd;
    state_load<LP, false>(S, start, a.d, w, lane);
    pair_zeros<false>(P, tid);
    if (tid < 2) wild[tid] = 0;
    if (tid < LP) first_wild[0][tid] = first_wild[1][tid] = kC;
    if (clock && p.c0 < p.c1) {
        decays(decs[p.c0 & 1], g, lane, &total);
        if (p.c0 + 1 < p.c1) g = decay_load(a, p, p.c0 + 1, lane);
    }

    for (int c = p.c0; c < p.c1; ++c) {
        const Decays &dec = decs[c & 1];
        const int rows = min(kC, p.len - c * kC);
        float term = 0.f, pairs = 0.f;
        if constexpr (MORE) {
            if (c > 0 && c % a.mark == 0 && p.split == 0) {
                float *at = a.marks + mark_at(a, p, c) * (LP * LP) + 4 * tid;
#pragma unroll
                for (int ct = 0; ct < O::CT; ++ct) *(DLRM_GLOBAL floatx4 *)(at + ct * 4 * THREADS) = S[ct];
            }
        }
        for (int h = 0; h < heads; ++h) {
            lds_barrier();  // the tiles before have been read
            if (h == 0) {
                zs.tame(first_wild[c & 1], &wild[c & 1]);
                ys.store(Ys), zs.store(Zs);
            }
            xs.store(Xs);
            if constexpr (MORE) ts.store(Ts);
            lds_barrier();
            load(h + 1 < heads ? c : c + 1, h + 1 < heads ? h + 1 : 0);
            if (clock && h == 0 && c + 1 < p.c1) {
                if (lane == 0) wild[~c & 1] = 0;
                for (int i = lane; i < LP; i += 64) first_wild[~c & 1][i] = kC;
                decays(decs[~c & 1], g, lane, &total);
                if (c + 2 < p.c1) g = decay_load(a, p, c + 2, lane);
            }
#pragma unroll
            for (int n = 0; n < (kTiles + O::WAVES - 1) / O::WAVES; ++n) {
                const int t = w + n * O::WAVES;
                if (t >= kTiles) break;
                const float sum = pair_tile<LP, false, false, GRAD == kEach ? kEach : kNone>(P, nullptr, dec, Xs, Ys, Ts, Zs, t, lane);
                if constexpr (GRAD == kEach) {
                    if (quad == 0) by_tile[t][ln] = sum;
                }
            }
            typename O::Out o;
            through_state<LP, PR>(o, S, Xs, lane);
            weigh<LP, MORE>(o, dec.from, Ts, by_wave[MORE ? w : 0], w, lane);
            lds_barrier();
            through_pairs<LP, false>(o, P, Zs, w, lane);
            if (__builtin_amdgcn_readfirstlane(wild[c & 1])) out_wild(o, first_wild[c & 1], w, lane);
            out_rows<LP>(o, Xs, a.out + ((p.row0 + c * kC) * a.Hq + h0 + h) * a.d, static_cast<int64_t>(a.Hq) * a.d, rows, a.d, a.scale, w,
                         lane);
            if (MORE && w == 0) {
                if constexpr (GRAD == kEach) {
                    const int ib = lane / 16;
                    for (int t = 0; t <= ib; ++t) pairs += by_tile[ib * (ib + 1) / 2 + t][ln];
                }
#pragma unroll
                for (int v = 0; v < O::WAVES; ++v) term += by_wave[v][lane];
            }
        }
        if (MORE && w == 0 && lane < rows) {
            const int64_t at = (p.split * a.Hkv + p.kvh) * a.N + p.row0 + c * kC + lane;
            a.terms[at] = term * a.scale;
            if constexpr (GRAD == kEach) a.pairs[at] = pairs * a.scale;
        }
        if (c + 1 == p.c1 && !a.last) break;  // nobody reads the state any more
        state_fade<LP>(S, dec.fade);
        state_grow<LP, UP>(S, Ys, Zs, dec.to, w, lane);
        if (__builtin_amdgcn_readfirstlane(wild[c & 1])) state_wild<LP>(S, first_wild[c & 1], w, lane);
    }
    if (a.last && p.c1 == p.chunks && p.split == 0)
        state_store<LP>(S, a.last + (static_cast<int64_t>(p.b) * a.Hkv + p.kvh) * dd, a.d, w, lane);
}

// What each run adds to the state, and how far it fades what was there.  REV: from the sequence's end, y and z
// the query heads' (all of a group add to one state).  Bound by reading the rows and writing the states, 64 KB for a head of 128:
// 3.5 TB/s (4 sequences of 2000 to 4096 in runs of two chunks, both directions in one launch, 21 us).
template <int LP, bool REV, int UP>
__device__ __forceinline__ void run_state(const Walk &a, uint16_t *Ys, uint16_t *Zs, Decays (&decs)[2]) {
    using O = Of<LP>;
    constexpr int THREADS = 64 * O::WAVES;
    const Part p = part_of(a);
    if (!p.any || p.chunks == 0 || (REV ? p.c0 == 0 : p.c1 == p.chunks)) return;  // what the last run adds is of no use
    const int lane = threadIdx.x & 63, w = static_cast<int>(wave_id());
    const int heads = REV ? a.group : 1, h0 = p.kvh * heads, n = p.c1 - p.c0;
    const uint16_t *yb = a.y.p + p.row0 * a.y.row + h0 * a.y.head;
    const uint16_t *zb = a.z.p + p.row0 * a.z.row + h0 * a.z.head;

    typename O::State S;
    state_load<LP, false>(S, nullptr, a.d, w, lane);
    Loader<LP, THREADS> ys(a.y.row, a.d), zs(a.z.row, a.d);
    const auto chunk = [&](int i) { return REV ? p.c1 - 1 - i : p.c0 + i; };
    const auto load = [&](int i, int h) {
        const int64_t row = static_cast<int64_t>(chunk(i)) * kC;
        const int rows = i < n ? p.len - chunk(i) * kC : 0;
        ys.load(yb + row * a.y.row + h * a.y.head, a.y.row, a.d, rows);
        zs.load(zb + row * a.z.row + h * a.z.head, a.z.row, a.d, rows);
    };
    double total = 0.0;
    float g = 0.f;
    if (w == 0) g = decay_load(a, p, chunk(0), lane);
    load(0, 0);
    if (w == 0) {
        decays(decs[0], g, lane, &total);
        if (n > 1) g = decay_load(a, p, chunk(1), lane);
    }
    for (int i = 0; i < n; ++i) {
        const Decays &dec = decs[i & 1];
        for (int h = 0; h < heads; ++h) {
            lds_barrier();
            ys.store(Ys), zs.store(Zs);
            lds_barrier();
            load(h + 1 < heads ? i : i + 1, h + 1 < heads ? h + 1 : 0);
            if (h == 0) {
                if (w == 0 && i + 1 < n) {
                    decays(decs[~i & 1], g, lane, &total);
                    if (i + 2 < n) g = decay_load(a, p, chunk(i + 2), lane);
                }
                state_fade<LP>(S, dec.fade);
            }
            state_grow<LP, UP>(S, Ys, Zs, REV ? dec.from : dec.to, w, lane);
        }
    }
    const int64_t at = p.slot * static_cast<int64_t>(a.Hkv) + p.kvh;
    state_store<LP>(S, a.start + at * a.d * a.d, a.d, w, lane);
    if (w == 0 && lane == 0) a.fade[at] = exp2_of(total);
}

template <int LP, int UP, bool BACK>
__global__ __launch_bounds__(Of<LP>::WAVES * 64, 4) void k_decay_runs(const Walk f, const Walk r) {
    __shared__ __attribute__((aligned(16))) uint16_t Ys[Of<LP>::TILE], Zs[Of<LP>::TILE];
    __shared__ __attribute__((aligned(16))) Decays decs[2];
    if (BACK && blockIdx.y == 0) run_state<LP, true, UP>(r, Ys, Zs, decs);  // the longer one first
    else run_state<LP, false, UP>(f, Ys, Zs, decs);
}

// The states at the runs' starts, in place of what the runs add, four elements a thread; sixteen runs are read at once, as
// each waits for the one before only in its sum.  Bound by reading and writing the states: 4.3 TB/s.
template <bool REV>
__device__ __forceinline__ void join(const Walk &a, uint32_t blocks) {
    const uint32_t id = blockIdx.x / blocks, part = blockIdx.x % blocks;
    const int b = static_cast<int>(id / a.Hkv), kvh = static_cast<int>(id % a.Hkv);
    const int64_t dd = static_cast<int64_t>(a.d) * a.d, e = (part * 64 + threadIdx.x) * int64_t(4);
    const int T = kC * a.run;
    const int r0 = offset_at(a, a.off, b, a.N), r1 = offset_at(a, a.off, b + 1, a.N);
    const int runs = (max(r1 - r0, 0) + T - 1) / T;
    if ((runs < 2 && !a.all_start) || e >= dd) return;
    const int64_t slot0 = r0 / T + b;
    const auto at = [&](int i) { return (slot0 + (REV ? runs - 1 - i : i)) * a.Hkv + kvh; };
    float *const states = a.start + e;
    floatx4 s = {0.f, 0.f, 0.f, 0.f};
    if (!REV && a.first) s = *reinterpret_cast<const floatx4 *>(a.first + id * dd + e);
    if (runs < 2) {
        *reinterpret_cast<floatx4 *>(states + (slot0 * a.Hkv + kvh) * dd) = s;
        return;
    }
    constexpr int AT_ONCE = 16;
    for (int i0 = 0; i0 + 1 < runs; i0 += AT_ONCE) {
        floatx4 add[AT_ONCE];
        float f[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
            if (i0 + i + 1 < runs) add[i] = *reinterpret_cast<const floatx4 *>(states + at(i0 + i) * dd), f[i] = a.fade[at(i0 + i)];
        // (run i's place takes its start, the last one's, which adds nothing that is wanted, too)
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            if (i0 + i + 1 >= runs) continue;
            if (i0 + i > 0 || a.all_start) *reinterpret_cast<floatx4 *>(states + at(i0 + i) * dd) = s;
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = fmaf(f[i], s[k], add[i][k]);
        }
    }
    *reinterpret_cast<floatx4 *>(states + at(runs - 1) * dd) = s;
}

__global__ __launch_bounds__(64) void k_decay_join(const Walk f, const Walk r, uint32_t blocks) {
    if (blockIdx.y == 0) join<false>(f, blocks);
    else join<true>(r, blocks);
}

// The sequences by their chunks, the most first: a counting sort by one workgroup.  (Which of two equal ones comes
// first is left to chance: nothing but the time goes by it.)  1024 sequences: 4.8 us, a launch and a chain of waits.
__global__ __launch_bounds__(1024) void k_decay_order(const Walk a, int32_t *order) {
    constexpr int CLASSES = 1024;
    __shared__ int32_t count[CLASSES], wave[16];
    const int t = threadIdx.x, lane = t & 63, w = static_cast<int>(wave_id());
    const auto class_of = [&](int b) {
        const int n = max(offset_at(a, a.off, b + 1, a.N) - offset_at(a, a.off, b, a.N), 0);
        return CLASSES - 1 - min((n + kC - 1) / kC, CLASSES - 1);
    };
    count[t] = 0;
    __syncthreads();
    for (int b = t; b < a.B; b += 1024) atomicAdd(&count[class_of(b)], 1);
    __syncthreads();
    const int mine = count[t];
    int upto = mine;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
        const int up = __shfl_up(upto, i);
        if (lane >= i) upto += up;
    }
    if (lane == 63) wave[w] = upto;
    __syncthreads();
    for (int v = 0; v < w; ++v) upto += wave[v];
    count[t] = upto - mine;
    __syncthreads();
    for (int b = t; b < a.B; b += 1024) order[atomicAdd(&count[class_of(b)], 1)] = b;
}

template <int LP>
int walk_lp(const Walk &a, int up, int grad, hipStream_t stream) {
    const dim3 grid(workgroups_of(a)), block(Of<LP>::WAVES * 64);
    if (grad == kEach) DLRM_LAUNCH("seq_decay_dq", (k_decay_walk<LP, 3, 3, kEach>), grid, block, 0, stream, a);
    else if (grad == kHead) DLRM_LAUNCH("seq_decay_dq", (k_decay_walk<LP, 3, 3, kHead>), grid, block, 0, stream, a);
    else if (up == 3) DLRM_LAUNCH("seq_decay_walk", (k_decay_walk<LP, 3, 1, kNone>), grid, block, 0, stream, a);
    else DLRM_LAUNCH("seq_decay_walk", (k_decay_walk<LP, 2, 1, kNone>), grid, block, 0, stream, a);
    return launch_status();
}

template <int LP>
void runs_lp(const Walk &f, const Walk *r, int up, hipStream_t stream) {
    const dim3 grid(workgroups_of(f), r ? 2 : 1), block(Of<LP>::WAVES * 64);
    if (r && up == 3) DLRM_LAUNCH("seq_decay_runs", (k_decay_runs<LP, 3, true>), grid, block, 0, stream, f, *r);
    else if (r) DLRM_LAUNCH("seq_decay_runs", (k_decay_runs<LP, 2, true>), grid, block, 0, stream, f, *r);
    else if (up == 3) DLRM_LAUNCH("seq_decay_runs", (k_decay_runs<LP, 3, false>), grid, block, 0, stream, f, f);
    else DLRM_LAUNCH("seq_decay_runs", (k_decay_runs<LP, 2, false>), grid, block, 0, stream, f, f);
}

}  // namespace

int run_states(const Walk &f, const Walk *r, int up, hipStream_t stream) {
    if (f.d <= 32) runs_lp<32>(f, r, up, stream);
    else if (f.d <= 64) runs_lp<64>(f, r, up, stream);
    else runs_lp<128>(f, r, up, stream);
    const uint32_t blocks = (static_cast<uint32_t>(f.d * f.d) / 4 + 63) / 64;
    DLRM_LAUNCH("seq_decay_join", k_decay_join, dim3(static_cast<uint32_t>(f.B) * f.Hkv * blocks, r ? 2 : 1), dim3(64), 0, stream, f, r ? *r : f, blocks);
    return launch_status();
}

int order_by_length(const Walk &a, int32_t *order, hipStream_t stream) {
    DLRM_LAUNCH("seq_decay_order", k_decay_order, dim3(1), dim3(1024), 0, stream, a, order);
    return launch_status();
}

int walk(const Walk &a, int up, int grad, hipStream_t stream) {
    if (a.d <= 32) return walk_lp<32>(a, up, grad, stream);
    if (a.d <= 64) return walk_lp<64>(a, up, grad, stream);
    return walk_lp<128>(a, up, grad, stream);
}

}  // namespace decay
}  // namespace seq
}  // namespace dlrm

extern "C" size_t dlrm_seq_decay_fwd_workspace_size(const dlrm_seq_decay *desc) {
    using namespace dlrm::seq::decay;
    Walk a;
    if (check(desc, true, &a) != DLRM_OK) return 0;
    const Cut c = cut_of(a, desc->max_len, false);
    return 256 + states_bytes(a, c) + order_bytes(a, c);
}

extern "C" int dlrm_seq_decay_fwd(const dlrm_seq_decay *desc, const float *state_in, float *state_out, uint16_t *o, void *workspace,
                                  size_t workspace_bytes, dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq::decay;
    Walk a;
    int rc = check(desc, true, &a);
    if (rc != DLRM_OK) return rc;
    if ((a.N > 0 && !o) || !aligned(o, 16) || !aligned(state_in, 16) || !aligned(state_out, 16)) return DLRM_ERR_INVALID_ARG;
    if (a.B == 0) return DLRM_OK;
    const Cut c = cut_of(a, desc->max_len, false);
    if ((c.run || c.order) && (!workspace || !aligned(workspace, 256) || workspace_bytes < dlrm_seq_decay_fwd_workspace_size(desc)))
        return DLRM_ERR_WORKSPACE;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    const int up = state_out ? 3 : 2;
    a.run = c.run, a.slots = static_cast<uint32_t>(c.slots);
    a.first = state_in, a.last = state_out, a.out = o;
    if (c.run) {
        a.start = static_cast<float *>(workspace);
        a.fade = a.start + c.slots * a.Hkv * a.d * a.d;
        a.all_start = state_in && state_in == state_out;
        rc = run_states(a, nullptr, up, stream);
    } else if (c.order) {
        int32_t *order = static_cast<int32_t *>(workspace);
        rc = order_by_length(a, order, stream);
        a.order = order;
    }
    if (rc != DLRM_OK) return rc;
    // in place, one workgroup reads and writes a whole sequence's state
    a.splits = state_in && state_in == state_out && !c.run ? 1 : splits_of(a, false);
    return walk(a, up, kNone, stream);
}
