// Attention of one new event a sequence over its cached keys and values (dlrm_seq.h).
//
// Bound by reading the cache once.  A workgroup takes one key/value head of one sequence, or a run
// of its visible keys where there are too few of them to fill the GPU, and up to 16 query heads
// that share it: each byte of the cache is read by one wavefront.  Each of the four wavefronts walks
// chunks of 32 keys with its own running maximum and sum; their results are joined at the end, those
// of several runs by a second kernel.  The products are 16x16x32 matrix instructions on transposed
// tiles, as in the forward: K goes from memory straight into the first operand, P^T stays in
// registers, and V passes through LDS, each wavefront's own, for the transposed read.  P is rounded to bf16
// for its product, as there.
//
// Measured: 32 sequences of 32768 to 65536, 8 heads of 128 over 1: 151 us, 5.3 TB/s, the rate of a large
// copy, and 12 for the join; 256 of 64 to 8192, 8 heads of 64 over 2: 48 us, 4.3 TB/s, and 6.6; one
// of 150 to 200, 4 heads of 32: 8.6 us, a chain of waits for memory.
#include <algorithm>

#include "seq.h"

namespace dlrm {
namespace seq {
namespace {

constexpr int kHeads = 16;  // query heads a workgroup: the columns of a product
constexpr int kWaves = 4;
constexpr int kChunk = 32;  // keys a wavefront takes at once
// Wavefronts a SIMD that the registers have to leave room for: unbound, heads of 64 took 150 and three
// fitted (256 of 64 to 8192, 8 heads over 2: 48.8 us, with four 47.4).
template <int DP>
constexpr int kOcc = DP == 32 ? 5 : DP == 64 ? 4 : 2;

__device__ __forceinline__ float max_quarters(float x) {  // over lanes l, l ^ 16, l ^ 32, l ^ 48
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float add_quarters(float x) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return add_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// part: [B][Hq][splits] rows of d floats, the runs' outputs; ml: their (maximum, sum)
template <int DP>
__global__ __launch_bounds__(kWaves * 64, kOcc<DP>) void k_seq_attn_decode(const Args a, const int splits, const int quantum, const bool splits_first,
                                                                 const int head_groups,
                                                                 uint16_t *o_out, float *part, float2 *ml) {
    constexpr int LP = DP, CH = LP / 8, STEPS = DP / 32, MB = DP / 16, VN = kChunk * CH / 64;
    union Lds {
        uint16_t v[kWaves][kChunk * kPitch<LP>];
        float o[kWaves][kHeads][DP];
    };
    __shared__ __attribute__((aligned(16))) Lds lds;
    __shared__ __attribute__((aligned(16))) int ids[kWaves][kChunk];
    __shared__ float top_s[kWaves][kHeads], sum_s[kWaves][kHeads], unit_s[kWaves][kHeads];
    __shared__ float bias_s[kHeads * DLRM_SEQ_MAX_BUCKETS];
    __shared__ int bounds_s[DLRM_SEQ_MAX_BUCKETS];

    const int split = splits_first ? blockIdx.x : blockIdx.y;
    uint32_t id = splits_first ? blockIdx.y : blockIdx.x;
    const int hg = static_cast<int>(id % head_groups);
    id /= head_groups;
    const int kvh = static_cast<int>(id % a.Hkv), b = static_cast<int>(id / a.Hkv);
    const int h0 = kvh * a.group + hg * kHeads, heads = min(kHeads, a.group - hg * kHeads);
    const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, quad = lane >> 4;
    const int w = static_cast<int>(wave_id());

    const int64_t row0 = offset_at(a, a.kv_begin, b, a.Nkv);
    const int klen = max(offset_at(a, a.kv_end, b, a.Nkv) - static_cast<int>(row0), 0);
    // the visible keys in a row: the first `skip` ones, then those from `start` on
    const int start = a.window ? max(0, klen - a.window) : 0;
    const int skip = min(a.sinks, start);
    const int seen = skip + klen - start;
    const int per = max(((seen + kChunk - 1) / kChunk + splits - 1) / splits * kChunk, quantum);
    const int v0 = min(static_cast<int64_t>(split) * per, static_cast<int64_t>(seen)), v1 = min(v0 + per, seen);
    if (splits > 1 && v0 >= v1) {  // a run without keys: the join passes it over
        if (tid < heads) ml[(static_cast<int64_t>(b) * a.Hq + h0 + tid) * splits + split] = make_float2(-kInf, 0.f);
        return;
    }

    const uint16_t *kb = a.k + row0 * a.k_row + kvh * a.k_head;
    const uint16_t *vb = a.v + row0 * a.v_row + kvh * a.v_head;

    floatx4 o[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) o[m] = floatx4{0.f, 0.f, 0.f, 0.f};
    float top = -kInf, sum = 0.f;
    float known = 0.f, share = 1.f, unit = 1.f;  // the sum, if known; what P is multiplied by; a unit of o in the sum's terms

    u32x4 kr[2][STEPS], vr[VN];
    const auto load = [&](int c) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int v = c + 16 * g + ln;
            const int64_t key = v < skip ? v : start + v - skip;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                kr[g][s] = u32x4{0, 0, 0, 0};
                const int col = 32 * s + 8 * quad;
                if (v < v1 && col < a.d) kr[g][s] = *(const DLRM_GLOBAL u32x4 *)(kb + key * a.k_row + col);
            }
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int at = i * 64 + lane, v = c + at / CH, col = at % CH * 8;
            const int64_t key = v < skip ? v : start + v - skip;
            vr[i] = u32x4{0, 0, 0, 0};
            if (v < v1 && col < a.d) vr[i] = *(const DLRM_GLOBAL u32x4 *)(vb + key * a.v_row + col);
        }
    };

    // the first chunk and the queries are on their way while the bias is fetched
    int c = v0 + w * kChunk;
    if (c < v1) load(c);
    for (int i = tid; i < a.buckets; i += kWaves * 64) bounds_s[i] = a.bounds[i];
    for (int i = tid; i < a.buckets * heads; i += kWaves * 64) bias_s[i] = a.bias[static_cast<int64_t>(h0) * a.buckets + i];
    __syncthreads();
    const float *my_bias = bias_s + (ln < heads ? ln * a.buckets : 0);
    const float far = a.buckets ? my_bias[a.buckets - 1] : 0.f;

    Frag qf[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        qf[s].q = u32x4{0, 0, 0, 0};
        const int c = 32 * s + 8 * quad;
        if (ln < heads && c < a.d) qf[s].q = *(const DLRM_GLOBAL u32x4 *)(a.q + b * a.q_row + (h0 + ln) * a.q_head + c);
    }
    // An output is a mean of its values and finite where they are, but sum P v before the division may not
    // be.  Where a head's o overflowed and its sum did not, the wavefront walks its keys again with that sum as
    // known: P / sum adds up to 1.
#pragma unroll 1
    for (int walk = 0;; ++walk) {
        for (; c < v1; c += kWaves * kChunk) {
            uint16_t *vt = lds.v[w];
            floatx4 s[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                s[g] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    Frag k;
                    k.q = kr[g][i];
                    s[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k.b, qf[i].b, s[g], 0, 0, 0);
                }
            }
            wave_lds_sync();  // the chunk before has been read
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const int at = i * 64 + lane;
                *reinterpret_cast<u32x4 *>(vt + at / CH * kPitch<LP> + at % CH * 8) = vr[i];
            }
            const int next = c + kWaves * kChunk;
            if (next < v1) load(next);

            // register r of block g: key c + 16 g + 4 quad + r (of those in a row)
            const int last_v = min(c + kChunk, v1) - 1;
            const int nearest = klen - 1 - (last_v < skip ? last_v : start + last_v - skip);
            if (!a.buckets || nearest >= a.last) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[g][r] = fmaf(s[g][r], a.scale, far);
            } else {
                if (lane < kChunk) {
                    const int v = c + lane;
                    ids[w][lane] = bucket_of(bounds_s, a.buckets, max(0, klen - 1 - (v < skip ? v : start + v - skip)));
                }
                wave_lds_sync();
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[g][r] = fmaf(s[g][r], a.scale, my_bias[ids[w][16 * g + 4 * quad + r]]);
            }
            if (c + kChunk > v1) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (c + 16 * g + 4 * quad + r >= v1) s[g][r] = -kInf;
            }
            float mx = s[0][0];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int r = 0; r < 4; ++r) mx = fmaxf(mx, s[g][r]);
            mx = fmaxf(max_quarters(mx), top);
            if (__any(mx > top)) {
                const float f = mx == -kInf ? 1.f : __builtin_amdgcn_exp2f((top - mx) * kLog2e);
                sum *= f;
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[m][r] *= f;
                top = mx;
            }
            const float ref = top == -kInf ? 0.f : top;
            Frag p;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s[g][r] = __builtin_amdgcn_exp2f((s[g][r] - ref) * kLog2e) * share;
                    sum += s[g][r];
                }
                p.w[2 * g] = pack_bf16(s[g][0], s[g][1]);
                p.w[2 * g + 1] = pack_bf16(s[g][2], s[g][3]);
            }
            wave_lds_sync();
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                // column 16 m + ln of the keys 4 quad + {0..3} and those 16 further on
                typedef __attribute__((address_space(3))) s16x4 *lds_t;
                Frag v;
                const int col = 16 * m + 4 * (ln & 3), row = 4 * quad + (ln >> 2);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const uint16_t *at = vt + (row + 16 * g) * kPitch<LP> + col;
                    v.h[g] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(at));
                }
                o[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v.b, p.b, o[m], 0, 0, 0);
            }
        }
        sum = add_quarters(sum);
        if (walk == 1) {
            if (share != 1.f) unit = known / sum, sum = known;
            break;
        }
        float any = sum;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) any += o[m][r];
        const bool over = max_quarters(ln < heads && !(fabsf(any) < kInf) && sum > 0.f && sum < kInf ? 1.f : 0.f) != 0.f;
        if (!__any(over)) break;
        known = sum, share = over ? 1.f / sum : 1.f, top = over ? top : -kInf, sum = 0.f;
#pragma unroll
        for (int m = 0; m < MB; ++m) o[m] = floatx4{0.f, 0.f, 0.f, 0.f};
        c = v0 + w * kChunk;
        load(c);
    }

    // join the wavefronts
    __syncthreads();
    if (quad == 0) top_s[w][ln] = top, sum_s[w][ln] = sum, unit_s[w][ln] = unit;
#pragma unroll
    for (int m = 0; m < MB; ++m) *reinterpret_cast<floatx4 *>(&lds.o[w][ln][16 * m + 4 * quad]) = o[m];
    __syncthreads();
    for (int i = tid; i < heads * (DP / 4); i += kWaves * 64) {
        const int hd = i / (DP / 4), col = i % (DP / 4) * 4;
        if (col >= a.d) continue;
        float mx = top_s[0][hd];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) mx = fmaxf(mx, top_s[v][hd]);
        float total = 0.f, f[kWaves];
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            const float t = top_s[v][hd];
            f[v] = t == -kInf ? 0.f : __builtin_amdgcn_exp2f((t - mx) * kLog2e);
            total += f[v] * sum_s[v][hd];
        }
        // divided before they are added: each may be near the largest number
        const float inv = total == 0.f ? 0.f : 1.f / total;
        floatx4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            const floatx4 y = *reinterpret_cast<const floatx4 *>(&lds.o[v][hd][col]);
            const float g = f[v] * unit_s[v][hd] * inv;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += g * y[e];
        }
        const int64_t row = static_cast<int64_t>(b) * a.Hq + h0 + hd;
        if (splits == 1) {
            *(DLRM_GLOBAL u32x2 *)(o_out + row * a.d + col) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        } else {
            *(DLRM_GLOBAL floatx4 *)(part + (row * splits + split) * a.d + col) = x;
            if (col == 0) ml[row * splits + split] = make_float2(mx, total);
        }
    }
}

// Joins the runs of a row: a workgroup a row, its wavefronts one run each in turn, so that all reads are
// under way at once; then the wavefronts' sums in order.
__global__ __launch_bounds__(256) void k_seq_decode_join(const float *part, const float2 *ml, int splits, int d, uint16_t *o) {
    __shared__ float2 sums[kWaves][64];
    __shared__ float factor[kWaves][64];
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 63, w = static_cast<int>(wave_id());
    const float2 t = lane < splits ? ml[row * splits + lane] : make_float2(-kInf, 0.f);
    float mx = t.x;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) mx = fmaxf(mx, __shfl_xor(mx, i));
    const float f = (t.x == -kInf ? 0.f : __builtin_amdgcn_exp2f((t.x - mx) * kLog2e)) * t.y;
    float total = f;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) total += __shfl_xor(total, i);
    float x = 0.f, y = 0.f;
    const float *p = part + row * splits * d + 2 * lane;
    factor[w][lane] = total == 0.f ? 0.f : f / total;
    wave_lds_sync();
#pragma unroll 16
    for (int s = w; s < splits; s += kWaves) {
        const float g = factor[w][s];
        if (g != 0.f && 2 * lane < d) {  // nothing was written for a run without keys
            const float2 v = *reinterpret_cast<const float2 *>(p + static_cast<int64_t>(s) * d);
            x = fmaf(g, v.x, x), y = fmaf(g, v.y, y);
        }
    }
    sums[w][lane] = make_float2(x, y);
    __syncthreads();
    if (w != 0 || 2 * lane >= d) return;
    x = y = 0.f;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) x += sums[v][lane].x, y += sums[v][lane].y;
    *reinterpret_cast<uint32_t *>(o + row * d + 2 * lane) = pack_bf16(x, y);
}

// How the keys of a sequence are split: into at most 64 runs of at least `quantum` keys.  A workgroup a
// sequence and key head is enough where there are many of one length; lengths differ, and the longest
// would end long after the others, so that some 4096 runs are aimed at, of 256 keys at least.
struct Split {
    int runs, quantum;
};

// Workgroups of a run of every sequence.
int64_t blocks_of(int64_t B, int32_t Hq, int32_t Hkv) { return B * Hkv * ((Hq / Hkv + kHeads - 1) / kHeads); }
constexpr int64_t kMostBlocks = (int64_t(1) << 24) - 1;  // of 256 threads: a launch holds fewer than 2^32 work-items

Split split_of(int64_t B, int32_t Hq, int32_t Hkv, int32_t window, int32_t sinks, int64_t max_kv_len) {
    const int64_t blocks = blocks_of(B, Hq, Hkv);
    int64_t seen = max_kv_len < (int64_t(1) << 30) ? max_kv_len : int64_t(1) << 30;
    if (window > 0 && static_cast<int64_t>(window) + sinks < seen) seen = static_cast<int64_t>(window) + sinks;
    int64_t quantum = (blocks * seen / 4096 + kChunk * kWaves - 1) / (kChunk * kWaves) * (kChunk * kWaves);
    quantum = quantum < 256 ? 256 : quantum > (1 << 20) ? 1 << 20 : quantum;
    const int64_t runs = (seen + quantum - 1) / quantum;
    return Split{static_cast<int>(runs < 1 ? 1 : runs > 64 ? 64 : runs), static_cast<int>(quantum)};
}

template <int DP>
int launch(const Args &a, const Split &sp, uint16_t *o, void *ws, hipStream_t stream) {
    const int splits = sp.runs;
    const int head_groups = (a.group + kHeads - 1) / kHeads;
    const int64_t rows = static_cast<int64_t>(a.B) * a.Hq, blocks = blocks_of(a.B, a.Hq, a.Hkv);
    float *part = static_cast<float *>(ws);
    float2 *ml = reinterpret_cast<float2 *>(part ? part + rows * splits * a.d : nullptr);
    // Many sequences: the first runs of all start first, as every one of them has keys; the runs that only
    // long sequences have fill in (256 sequences of 64 to 8192: 82 -> 48 us).  Few: a sequence's runs side
    // by side, as neighbours in memory (32 of up to 65536: 166 -> 152 us).
    const bool splits_first = blocks < 256;
    const dim3 grid = splits_first ? dim3(splits, static_cast<uint32_t>(blocks)) : dim3(static_cast<uint32_t>(blocks), splits);
    DLRM_LAUNCH("seq_attn_decode", (k_seq_attn_decode<DP>), grid, dim3(kWaves * 64), 0, stream, a,
                splits, sp.quantum, splits_first, head_groups, o, part, ml);
    for (int64_t row0 = 0; splits > 1 && row0 < rows; row0 += kMostBlocks)
        DLRM_LAUNCH("seq_decode_join", k_seq_decode_join, dim3(static_cast<uint32_t>(std::min(rows - row0, kMostBlocks))), dim3(256),
                    0, stream, static_cast<const float *>(part + row0 * splits * a.d),
                    static_cast<const float2 *>(ml + row0 * splits), splits, a.d, o + row0 * a.d);
    return launch_status();
}

}  // namespace
}  // namespace seq
}  // namespace dlrm

extern "C" size_t dlrm_seq_attn_decode_workspace_size(int64_t B, int32_t Hq, int32_t Hkv, int32_t d, int32_t window,
                                                      int32_t sinks, int64_t max_kv_len) {
    using namespace dlrm::seq;
    if (B < 0 || B >= (1 << 24) || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 4096 || d < 1 || d > 128 || window < 0 || sinks < 0 ||
        max_kv_len < 0 || blocks_of(B, Hq, Hkv) > kMostBlocks)
        return 0;
    const int splits = split_of(B, Hq, Hkv, window, sinks, max_kv_len).runs;
    return 256 + (splits > 1 ? static_cast<size_t>(B) * Hq * splits * (d + 2) * 4 : 0);
}

extern "C" int dlrm_seq_attn_decode(const dlrm_seq_attn *desc, int64_t max_kv_len, uint16_t *o, void *workspace,
                                    size_t workspace_bytes, dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq;
    Args a;
    const int rc = check_attn(desc, false, &a);
    if (rc != DLRM_OK) return rc;
    if (a.Nq != a.B || max_kv_len < 0) return DLRM_ERR_INVALID_ARG;
    if (a.B == 0) return DLRM_OK;
    if (!o || !aligned(o, 16)) return DLRM_ERR_INVALID_ARG;
    if (blocks_of(a.B, a.Hq, a.Hkv) > kMostBlocks) return DLRM_ERR_UNSUPPORTED;
    const Split sp = split_of(a.B, a.Hq, a.Hkv, a.window, a.sinks, max_kv_len);
    if (sp.runs > 1 && (!workspace || !aligned(workspace, 256) ||
                       workspace_bytes < dlrm_seq_attn_decode_workspace_size(a.B, a.Hq, a.Hkv, a.d, a.window, a.sinks, max_kv_len)))
        return DLRM_ERR_WORKSPACE;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    if (a.d <= 32) return launch<32>(a, sp, o, workspace, stream);
    if (a.d <= 64) return launch<64>(a, sp, o, workspace, stream);
    return launch<128>(a, sp, o, workspace, stream);
}
