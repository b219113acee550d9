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
        if (slot_count(a->N, a->B, kC) * a->Hkv > (int64_t(1) << 23)) return DLRM_ERR_UNSUPPORTED;
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

// Workgroups that fill the GPU.
static int64_t places_of(int32_t d) { return d <= 32 ? 1536 : d <= 64 ? 1024 : 512; }

// A sequence and key head a workgroup is enough where there are many; where few are long, they are cut into
// runs, whose states at the start are made first from k and v alone.
Cut cut_of(const Walk &a, int64_t max_len) {
    const int64_t longest = std::min(max_len, a.N), chunks = (longest + kC - 1) / kC;
    const int64_t all = slot_count(a.N, a.B, kC) * a.Hkv, places = places_of(a.d);
    int64_t share = std::max<int64_t>(4, (all + places - 1) / places);  // chunks for each place
    if (share > 8) share = (share + 7) / 8 * 8;
    const bool many = a.B * static_cast<int64_t>(a.Hkv) * 16 >= (int64_t(1) << 24);  // more than a launch of k_decay_join holds
    Cut c;
    c.run = chunks > 2 * share && !many ? static_cast<int32_t>(share) : 0;
    c.slots = c.run ? slot_count(a.N, a.B, kC * c.run) : a.B;
    return c;
}

int64_t state_floats(const Walk &a, const Cut &c) { return c.run ? c.slots * a.Hkv * (static_cast<int64_t>(a.d) * a.d + 1) : 0; }

int splits_of(const Walk &a) {
    int n = 1;
    while (n < a.group && static_cast<int64_t>(a.slots) * a.Hkv * n < places_of(a.d)) {
        do ++n;
        while (a.group % n != 0);
    }
    return n;
}

namespace {

template <int LP, int UP, int PR, int GRAD>
__global__ __launch_bounds__(Of<LP>::WAVES * 64, LP == 128 ? (GRAD ? 1 : 2) : LP == 64 ? (GRAD ? 3 : 4) : GRAD ? 2 : 3) void k_decay_walk(const Walk a) {
    constexpr bool MORE = GRAD != kNone;
    using O = Of<LP>;
    constexpr int THREADS = 64 * O::WAVES;
    __shared__ __attribute__((aligned(16))) uint16_t Xs[O::TILE], Ys[O::TILE], Zs[O::TILE], P[kC * kPP];
    __shared__ __attribute__((aligned(16))) Decays decs[2];
    __shared__ __attribute__((aligned(16))) uint16_t Ts[MORE ? O::TILE : 8];
    __shared__ float by_wave[MORE ? O::WAVES : 1][kC], by_tile[GRAD == kEach ? kTiles : 1][16];

    const Part p = part_of(a, xcd_contiguous(blockIdx.x, gridDim.x));
    if (!p.any) return;
    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, quad = lane >> 4;
    const int w = static_cast<int>(wave_id());
    const int heads = a.group / a.splits, h0 = p.kvh * a.group + p.split * heads;
    const uint16_t *xb = a.x.p + p.row0 * a.x.row + h0 * a.x.head;
    const uint16_t *yb = a.y.p + p.row0 * a.y.row + p.kvh * a.y.head;
    const uint16_t *zb = a.z.p + p.row0 * a.z.row + p.kvh * a.z.head;
    const uint16_t *tb = MORE ? a.t.p + p.row0 * a.t.row + h0 * a.t.head : nullptr;

    Stage<LP, THREADS> xs(a.x.row, a.d), ys(a.y.row, a.d), zs(a.z.row, a.d), ts(MORE ? a.t.row : 0, a.d);
    const auto load_yz = [&](int c) {
        ys.load(yb, a.y.row, a.d, c * kC, 0, p.len, 0);
        zs.load(zb, a.z.row, a.d, c * kC, 0, p.len, 0);
    };
    const auto load_x = [&](int c, int h) {
        xs.load(xb + h * a.x.head, a.x.row, a.d, c * kC, 0, p.len, 0);
        if constexpr (MORE) ts.load(tb + h * a.t.head, a.t.row, a.d, c * kC, 0, p.len, 0);
    };
    const bool clock = w == O::WAVES - 1;  // the wavefront that works out the next chunk's decays: it has the fewest tiles
    float g = 0.f;
    double total = 0.0;
    if (p.c0 < p.c1) {
        if (clock) g = decay_load(a, p, p.c0, lane);
        load_yz(p.c0), load_x(p.c0, 0);
    }
    typename O::State S;
    const int64_t dd = static_cast<int64_t>(a.d) * a.d;
    state_load<LP, false>(S, a.start ? a.start + ((a.run ? p.slot : p.b) * static_cast<int64_t>(a.Hkv) + p.kvh) * dd : nullptr, a.d, w, lane);
    pair_zeros<false>(P, tid);
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
                float *at = a.marks + ((p.row0 / (kC * a.mark) + p.b + c / a.mark) * a.Hkv + p.kvh) * (LP * LP) + 4 * tid;
#pragma unroll
                for (int i = 0; i < O::NB * O::CT; ++i) *(DLRM_GLOBAL floatx4 *)(at + i * 4 * THREADS) = S[i / O::CT][i % O::CT];
            }
        }
        for (int h = 0; h < heads; ++h) {
            lds_barrier();  // the tiles before have been read
            if (h == 0) tile_store(ys, Ys), tile_store(zs, Zs);
            tile_store(xs, Xs);
            if constexpr (MORE) tile_store(ts, Ts);
            lds_barrier();
            if (h + 1 < heads) load_x(c, h + 1);
            else if (c + 1 < p.c1) load_yz(c + 1), load_x(c + 1, 0);
            if (clock && h == 0 && c + 1 < p.c1) {
                decays(decs[~c & 1], g, lane, &total);
                if (c + 2 < p.c1) g = decay_load(a, p, c + 2, lane);
            }
#pragma unroll 1
            for (int t = w; t < kTiles; t += O::WAVES) {
                int jb, ib;
                tile_of<false>(t, &jb, &ib);
                const auto t_row = [&](int s) {
                    Frag f;
                    f.q = *reinterpret_cast<const u32x4 *>(Ts + (16 * ib + ln) * kPitch<LP> + 8 * quad + 32 * s);
                    return f;
                };
                const float sum = pair_tile<LP, false, GRAD == kEach ? kEach : kNone>(P, dec, Xs, Ys, t_row, Zs, jb, ib, lane);
                if constexpr (GRAD == kEach) {
                    if (quad == 0) by_tile[t][ln] = sum;
                }
            }
            typename O::Out o;
            through_state<LP, PR>(o, S, Xs, lane);
            weigh<LP, MORE>(o, dec.from, Ts, by_wave[MORE ? w : 0], w, lane);
            lds_barrier();
            typename O::Out before;
#pragma unroll
            for (int i = 0; i < O::NB * 4; ++i) before[i / 4][i % 4] = o[i / 4][i % 4];
            through_pairs<LP, false>(o, P, Zs, w, lane);
            float any = 0.f;
#pragma unroll
            for (int i = 0; i < O::NB * 4; ++i) {
                const floatx4 x = o[i / 4][i % 4];
                any += (x[0] + x[1]) + (x[2] + x[3]);
            }
            if (__any(!(fabsf(any) < kInf))) {
                // an infinity or NaN in z reaches the rows before it (0 * NaN in a product): once more, with its rows apart
#pragma unroll
                for (int i = 0; i < O::NB * 4; ++i) o[i / 4][i % 4] = before[i / 4][i % 4];
                through_pairs_apart<LP>(o, P, Zs, w, lane);
            }
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
    }
    if (a.last && p.c1 == p.chunks && p.split == 0)
        state_store<LP>(S, a.last + (static_cast<int64_t>(p.b) * a.Hkv + p.kvh) * dd, a.d, w, lane);
}

// What each run adds to the state, and how far it fades what was there.  REV: from the sequence's end, y and z
// the query heads' (all of a group add to one state).
template <int LP, bool REV, int UP>
__global__ __launch_bounds__(Of<LP>::WAVES * 64, LP == 128 ? 2 : 4) void k_decay_runs(const Walk a, float *states) {
    using O = Of<LP>;
    constexpr int THREADS = 64 * O::WAVES;
    __shared__ __attribute__((aligned(16))) uint16_t Ys[O::TILE], Zs[O::TILE];
    __shared__ __attribute__((aligned(16))) Decays decs[2];

    const Part p = part_of(a, xcd_contiguous(blockIdx.x, gridDim.x));
    if (!p.any || p.chunks == 0 || (REV ? p.c0 == 0 : p.c1 == p.chunks)) return;  // what the last run adds is of no use
    const int lane = threadIdx.x & 63, w = static_cast<int>(wave_id());
    const int heads = REV ? a.group : 1, h0 = p.kvh * heads, n = p.c1 - p.c0;
    const uint16_t *yb = a.y.p + p.row0 * a.y.row + h0 * a.y.head;
    const uint16_t *zb = a.z.p + p.row0 * a.z.row + h0 * a.z.head;

    typename O::State S;
    state_load<LP, false>(S, nullptr, a.d, w, lane);
    Stage<LP, THREADS> ys(a.y.row, a.d), zs(a.z.row, a.d);
    const auto chunk = [&](int i) { return REV ? p.c1 - 1 - i : p.c0 + i; };
    const auto load = [&](int i, int h) {
        ys.load(yb + h * a.y.head, a.y.row, a.d, chunk(i) * kC, 0, p.len, 0);
        zs.load(zb + h * a.z.head, a.z.row, a.d, chunk(i) * kC, 0, p.len, 0);
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
            tile_store(ys, Ys), tile_store(zs, Zs);
            lds_barrier();
            if (h + 1 < heads) load(i, h + 1);
            else if (i + 1 < n) load(i + 1, 0);
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
    state_store<LP>(S, states + at * a.d * a.d, a.d, w, lane);
    if (w == 0 && lane == 0) a.fade[at] = __builtin_amdgcn_exp2f(static_cast<float>(total));
}

// The states at the runs' starts, in place of what the runs add: four elements a thread.
template <bool REV>
__global__ __launch_bounds__(256) void k_decay_join(const Walk a, const float *first, float *states, uint32_t blocks) {
    const uint32_t id = blockIdx.x / blocks, part = blockIdx.x % blocks;
    const int b = static_cast<int>(id / a.Hkv), kvh = static_cast<int>(id % a.Hkv);
    const int64_t dd = static_cast<int64_t>(a.d) * a.d, e = (part * 256 + threadIdx.x) * int64_t(4);
    if (e >= dd) return;
    const int T = kC * a.run;
    const int r0 = offset_at(a, a.off, b, a.N), r1 = offset_at(a, a.off, b + 1, a.N);
    const int runs = (max(r1 - r0, 0) + T - 1) / T;
    const int64_t slot0 = r0 / T + b;
    floatx4 s = {0.f, 0.f, 0.f, 0.f};
    if (first) s = *reinterpret_cast<const floatx4 *>(first + id * dd + e);
#pragma unroll 4
    for (int i = 0; i < max(runs, 1); ++i) {
        const int64_t at = (slot0 + (REV ? runs - 1 - i : i)) * a.Hkv + kvh;
        floatx4 *p = reinterpret_cast<floatx4 *>(states + at * dd + e);
        if (i + 1 < runs) {
            const floatx4 add = *p;
            const float f = a.fade[at];
            *p = s;
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = fmaf(f, s[k], add[k]);
        } else if (!REV || runs > 0) {
            *p = s;
        }
    }
}

uint32_t grid_of(const Walk &a) { return round_up_xcd(static_cast<uint64_t>(a.slots) * a.Hkv * a.splits); }

template <int LP>
int walk_lp(const Walk &a, int up, int grad, hipStream_t stream) {
    const dim3 grid(grid_of(a)), block(Of<LP>::WAVES * 64);
    if (grad == kEach) DLRM_LAUNCH("seq_decay_dq", (k_decay_walk<LP, 3, 3, kEach>), grid, block, 0, stream, a);
    else if (grad == kHead) DLRM_LAUNCH("seq_decay_dq", (k_decay_walk<LP, 3, 3, kHead>), grid, block, 0, stream, a);
    else if (up == 3) DLRM_LAUNCH("seq_decay_walk", (k_decay_walk<LP, 3, 1, kNone>), grid, block, 0, stream, a);
    else DLRM_LAUNCH("seq_decay_walk", (k_decay_walk<LP, 2, 1, kNone>), grid, block, 0, stream, a);
    return launch_status();
}

template <int LP, bool REV>
void runs_lp(const Walk &a, int up, float *states, hipStream_t stream) {
    const dim3 grid(grid_of(a)), block(Of<LP>::WAVES * 64);
    if (up == 3) DLRM_LAUNCH("seq_decay_runs", (k_decay_runs<LP, REV, 3>), grid, block, 0, stream, a, states);
    else DLRM_LAUNCH("seq_decay_runs", (k_decay_runs<LP, REV, 2>), grid, block, 0, stream, a, states);
}

template <bool REV>
int run_states_of(const Walk &a, int up, const float *first, float *states, hipStream_t stream) {
    if (a.d <= 32) runs_lp<32, REV>(a, up, states, stream);
    else if (a.d <= 64) runs_lp<64, REV>(a, up, states, stream);
    else runs_lp<128, REV>(a, up, states, stream);
    const uint32_t blocks = (static_cast<uint32_t>(a.d * a.d) / 4 + 255) / 256;
    const int64_t all = static_cast<int64_t>(a.B) * a.Hkv * blocks;
    DLRM_LAUNCH("seq_decay_join", (k_decay_join<REV>), dim3(static_cast<uint32_t>(all)), dim3(256), 0, stream, a, first, states, blocks);
    return launch_status();
}

}  // namespace

int run_states(const Walk &a, const Cut &c, bool reversed, int up, const float *first, float *states, hipStream_t stream) {
    Walk r = a;
    r.splits = 1;
    r.run = c.run, r.slots = static_cast<uint32_t>(c.slots);
    r.fade = states + c.slots * a.Hkv * a.d * a.d;
    return reversed ? run_states_of<true>(r, up, first, states, stream) : run_states_of<false>(r, up, first, states, stream);
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
    return 256 + 4 * static_cast<size_t>(state_floats(a, cut_of(a, desc->max_len)));
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
    const Cut c = cut_of(a, desc->max_len);
    if (c.run && (!workspace || !aligned(workspace, 256) || workspace_bytes < dlrm_seq_decay_fwd_workspace_size(desc)))
        return DLRM_ERR_WORKSPACE;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    const int up = state_out ? 3 : 2;
    a.run = c.run, a.slots = static_cast<uint32_t>(c.slots);
    a.start = state_in, a.last = state_out, a.out = o;
    if (c.run) {
        float *states = static_cast<float *>(workspace);
        rc = run_states(a, c, false, up, state_in, states, stream);
        if (rc != DLRM_OK) return rc;
        a.start = states;
    }
    a.splits = splits_of(a);
    return walk(a, up, kNone, stream);
}
