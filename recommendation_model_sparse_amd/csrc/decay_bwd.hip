// Linear attention with a decay, backward (dlrm_seq_decay.h): dq by the forward walk on (do, v, k), dk and dv by
// a walk in reverse time, dg from both.
#include "decay.h"

namespace dlrm {
namespace seq {
namespace decay {
namespace {

// dk and dv in one walk from a sequence's end: two teams of wavefronts over the same tiles, the first for dv
// (x = k, y = q, z = do), the second for dk (x = v, y = do, z = q); the state of the second is the first's, transposed.
// a.x, a.y, a.z, a.t: k, q, do, v; a.out: dv, a.out2: dk; a.start: the first team's states.
template <int LP, int UP, int PR, bool MORE>
__global__ __launch_bounds__(LP * 4, 2) void k_decay_back(const Walk a) {
    using O = Of<LP>;
    constexpr int THREADS = 128 * O::WAVES;
    __shared__ __attribute__((aligned(16))) uint16_t Ks[O::TILE], Vs[O::TILE], Qs[O::TILE], Ds[O::TILE], Ps[2][kC * kPP];
    __shared__ __attribute__((aligned(16))) Decays dec;
    __shared__ float fade_s, by_wave[MORE ? O::WAVES : 1][kC], by_tile[MORE ? 3 : 1][32];

    const Part p = part_of(a, xcd_contiguous(blockIdx.x, gridDim.x));
    if (!p.any) return;
    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, half = lane >> 5;
    const int team = static_cast<int>(wave_id()) / O::WAVES, w = static_cast<int>(wave_id()) % O::WAVES;
    const int h0 = p.kvh * a.group;
    const uint16_t *kb = a.x.p + p.row0 * a.x.row + p.kvh * a.x.head;
    const uint16_t *vb = a.t.p + p.row0 * a.t.row + p.kvh * a.t.head;
    const uint16_t *qb = a.y.p + p.row0 * a.y.row + h0 * a.y.head;
    const uint16_t *db = a.z.p + p.row0 * a.z.row + h0 * a.z.head;
    const uint16_t *const xt = team ? Vs : Ks, *const yt = team ? Ds : Qs, *const zt = team ? Qs : Ds;
    uint16_t *const P = Ps[team];

    f32x16 S[O::CT];
    const float *start = a.start ? a.start + (p.slot * static_cast<int64_t>(a.Hkv) + p.kvh) * a.d * a.d : nullptr;
    if (team) state_load<LP, true>(S, start, a.d, w, lane);
    else state_load<LP, false>(S, start, a.d, w, lane);

    Stage<LP, THREADS> ks(a.x.row, a.d), vs(a.t.row, a.d), qs(a.y.row, a.d), ds(a.z.row, a.d);
    float g = 0.f;
    const auto load_kv = [&](int c) {
        ks.load(kb, a.x.row, a.d, c * kC, 0, p.len, 0);
        vs.load(vb, a.t.row, a.d, c * kC, 0, p.len, 0);
        if (tid < 64) g = decay_load(a, p, c, lane);
    };
    const auto load_q = [&](int c, int h) {
        qs.load(qb + h * a.y.head, a.y.row, a.d, c * kC, 0, p.len, 0);
        ds.load(db + h * a.z.head, a.z.row, a.d, c * kC, 0, p.len, 0);
    };
    if (p.c0 < p.c1) load_kv(p.c1 - 1), load_q(p.c1 - 1, 0);

    double total = 0.0;
    for (int c = p.c1 - 1; c >= p.c0; --c) {
        const int rows = min(kC, p.len - c * kC);
        f32x16 o[2];
        float term = 0.f;
        for (int h = 0; h < a.group; ++h) {
            __syncthreads();  // the tiles before have been read
            if (h == 0) {
                ks.store(Ks), vs.store(Vs);
                if (tid < 64) {
                    const float f = decays(dec, g, lane, &total);
                    if (lane == 0) fade_s = f;
                }
            }
            qs.store(Qs), ds.store(Ds);
            __syncthreads();
            if (h + 1 < a.group) load_q(c, h + 1);
            else if (c > p.c0) load_kv(c - 1), load_q(c - 1, 0);

            for (int t = w; t < 3; t += O::WAVES) {
                int jb, ib;
                tile_of<true>(t, &jb, &ib);
                const auto k_row = [&](int s) {
                    Frag f;
                    read_row(f, Ks + row_base<LP>(32 * ib + ln, half), s);
                    return f;
                };
                if (MORE && team == 1) {
                    const float sum = pair_tile<LP, true, MORE>(P, dec, xt, yt, k_row, Qs, jb, ib, lane);
                    if (half == 0) by_tile[t][ln] = sum;
                } else {
                    pair_tile<LP, true, false>(P, dec, xt, yt, k_row, nullptr, jb, ib, lane);
                }
            }
            if (h == 0) {
                through_state<LP, PR>(o, S, xt, lane);
#pragma unroll
                for (int ib = 0; ib < 2; ++ib) {
                    const float f = dec.to[32 * ib + ln];
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[ib][r] *= f;
                    if (MORE && team == 1) {
                        float sum = 0.f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const u32x2 v = *reinterpret_cast<const u32x2 *>(Ks + (32 * ib + ln) * kPitch<LP> + 32 * w + 8 * k + 4 * half);
                            sum += o[ib][4 * k] * bf16_lo(v.x) + o[ib][4 * k + 1] * bf16_hi(v.x);
                            sum += o[ib][4 * k + 2] * bf16_lo(v.y) + o[ib][4 * k + 3] * bf16_hi(v.y);
                        }
                        sum = add_halves(sum);
                        if (half == 0) by_wave[w][32 * ib + ln] = sum;
                    }
                }
                const float f = fade_s;
#pragma unroll
                for (int ct = 0; ct < O::CT; ++ct)
#pragma unroll
                    for (int r = 0; r < 16; ++r) S[ct][r] *= f;
            }
            __syncthreads();
            through_pairs<LP, true>(o, P, zt, w, lane);
            state_grow<LP, UP>(S, yt, zt, dec.from, w, lane);
            if (MORE && tid < 64) {
                float sum = lane < 32 ? by_tile[0][ln] + by_tile[1][ln] : by_tile[2][ln];
                if (h == 0) {
#pragma unroll
                    for (int v = 0; v < O::WAVES; ++v) sum += by_wave[v][lane];
                }
                term += sum;
            }
        }
        out_rows<LP>(o, (team ? a.out2 : a.out) + ((p.row0 + c * kC) * a.Hkv + p.kvh) * a.d, static_cast<int64_t>(a.Hkv) * a.d, rows, a.d,
                     a.scale, w, lane);
        if (MORE && tid < 64 && lane < rows) a.terms[p.kvh * a.N + p.row0 + c * kC + lane] = term * a.scale;
    }
}

// dg_t = the sum over i >= t of a sequence's <q_i, dq_i> - <k_i, dk_i>, in fp64: a workgroup a sequence and key head, 1024
// events at once from its end.  Where one decay stands for a head, the sum over t instead.
__global__ __launch_bounds__(256) void k_decay_dg(const Walk a, const float *plus, const float *minus, float *dg, double *sums) {
    __shared__ double part[4];
    const int b = static_cast<int>(blockIdx.x / a.Hkv), kvh = static_cast<int>(blockIdx.x % a.Hkv);
    const int64_t r0 = offset_at(a, a.off, b, a.N);
    const int len = max(offset_at(a, a.off, b + 1, a.N) - static_cast<int>(r0), 0);
    const int lane = threadIdx.x & 63, w = static_cast<int>(wave_id());
    const float *pp = plus + kvh * a.N + r0, *mp = minus + kvh * a.N + r0;
    double carry = 0.0, all = 0.0;
    for (int end = len; end > 0; end -= 1024) {
        // thread i has the events end - 1 - 4 i and the three before
        const int t0 = end - 1 - 4 * static_cast<int>(threadIdx.x);
        double x[4], s = 0.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (t0 - k >= 0) s += static_cast<double>(pp[t0 - k]) - static_cast<double>(mp[t0 - k]);
            x[k] = s;
        }
        double before = s;
#pragma unroll
        for (int i = 1; i < 64; i <<= 1) {
            const double up = __shfl_up(before, i);
            if (lane >= i) before += up;
        }
        __syncthreads();
        if (lane == 63) part[w] = before;
        __syncthreads();
        double base = carry + before - s;
        for (int v = 0; v < 4; ++v) {
            if (v < w) base += part[v];
            carry += part[v];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (t0 - k < 0) continue;
            const float g = a.g[(r0 + t0 - k) * a.g_row + kvh];
            const double d = g > 0.f ? 0.0 : base + x[k];
            if (sums) all += d;
            else dg[(r0 + t0 - k) * a.Hkv + kvh] = static_cast<float>(d);
        }
    }
    if (!sums) return;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) all += __shfl_xor(all, i);
    __syncthreads();
    if (lane == 0) part[w] = all;
    __syncthreads();
    if (threadIdx.x == 0) sums[static_cast<int64_t>(kvh) * a.B + b] = part[0] + part[1] + part[2] + part[3];
}

// dg of one decay a head: over the sequences, in a fixed order.
__global__ __launch_bounds__(256) void k_decay_dg_join(const double *sums, int32_t B, float *dg) {
    __shared__ double part[4];
    const int lane = threadIdx.x & 63, w = static_cast<int>(wave_id());
    double s = 0.0;
    for (int i = threadIdx.x; i < B; i += 256) s += sums[static_cast<int64_t>(blockIdx.x) * B + i];
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) s += __shfl_xor(s, i);
    if (lane == 0) part[w] = s;
    __syncthreads();
    if (threadIdx.x == 0) dg[blockIdx.x] = static_cast<float>(part[0] + part[1] + part[2] + part[3]);
}

template <int LP>
int back(const Walk &a, bool more, hipStream_t stream) {
    const dim3 grid(round_up_xcd(static_cast<uint64_t>(a.slots) * a.Hkv)), block(LP * 4);
    if (more) DLRM_LAUNCH("seq_decay_dkv", (k_decay_back<LP, 3, 3, true>), grid, block, 0, stream, a);
    else DLRM_LAUNCH("seq_decay_dkv", (k_decay_back<LP, 2, 1, false>), grid, block, 0, stream, a);
    return launch_status();
}

// Bytes: the runs' states, both terms of dg, the sequences' sums.
struct Room {
    size_t states, terms, sums;
};
Room room_of(const Walk &a, const Cut &c) {
    const auto whole = [](size_t n) { return (n + 255) / 256 * 256; };
    return Room{whole(4 * static_cast<size_t>(state_floats(a, c))), whole(8 * static_cast<size_t>(a.N) * a.Hkv),
                whole(8 * static_cast<size_t>(a.B) * a.Hkv)};
}

}  // namespace
}  // namespace decay
}  // namespace seq
}  // namespace dlrm

extern "C" size_t dlrm_seq_decay_bwd_workspace_size(const dlrm_seq_decay *desc) {
    using namespace dlrm::seq::decay;
    Walk a;
    if (check(desc, true, &a) != DLRM_OK) return 0;
    const Room r = room_of(a, cut_of(a, desc->max_len));
    return 256 + r.states + r.terms + r.sums;
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
    const bool more = dg != nullptr, by_head = more && a.g_row == 0;
    const Cut c = cut_of(a, desc->max_len);
    const Room room = room_of(a, c);
    char *ws = static_cast<char *>(workspace);
    float *states = reinterpret_cast<float *>(ws), *terms = reinterpret_cast<float *>(ws + room.states);
    double *sums = reinterpret_cast<double *>(ws + room.states + room.terms);
    const int up = more ? 3 : 2;
    const Heads q = a.x, k = a.y, v = a.z, d = {dout, static_cast<int64_t>(a.Hq) * a.d, a.d};
    a.run = c.run, a.slots = static_cast<uint32_t>(c.slots);
    if (a.N > 0 && a.B > 0) {
        a.x = d, a.y = v, a.z = k, a.t = q;
        a.out = dq, a.terms = terms;
        if (c.run) {
            rc = run_states(a, c, false, up, nullptr, states, stream);
            if (rc != DLRM_OK) return rc;
            a.start = states;
        }
        rc = walk(a, up, more, stream);
        if (rc != DLRM_OK) return rc;
        a.x = k, a.y = q, a.z = d, a.t = v;
        a.out = dv, a.out2 = dk, a.terms = terms + a.N * a.Hkv;
        if (c.run) {
            rc = run_states(a, c, true, up, nullptr, states, stream);
            if (rc != DLRM_OK) return rc;
        }
        rc = a.d <= 32 ? back<32>(a, more, stream) : a.d <= 64 ? back<64>(a, more, stream) : back<128>(a, more, stream);
        if (rc != DLRM_OK) return rc;
        if (more)
            DLRM_LAUNCH("seq_decay_dg", k_decay_dg, dim3(static_cast<uint32_t>(a.B) * a.Hkv), dim3(256), 0, stream, a,
                        static_cast<const float *>(terms), static_cast<const float *>(terms + a.N * a.Hkv), dg, by_head ? sums : nullptr);
    }
    if (by_head)
        DLRM_LAUNCH("seq_decay_dg_join", k_decay_dg_join, dim3(a.Hkv), dim3(256), 0, stream, static_cast<const double *>(sums),
                    a.N > 0 ? a.B : 0, dg);
    return launch_status();
}
