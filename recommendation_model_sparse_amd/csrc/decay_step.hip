// Linear attention with a decay, one event of each sequence (dlrm_seq_decay.h).
//
// Bound by reading and writing the states once.  A workgroup takes one key head's state of one sequence: each
// thread four neighbouring columns of some of its rows, which stay in registers for all query heads that share it.
// Measured: 512 sequences, 4 states of 128 x 128 each, 41 us, 272 MB at 6.6 TB/s (part of the states is still in the
// caches from the call before; with other states in between 59 us, 4.6); one sequence, 4 of 32 x 32, 3.8 us, a launch
// and three waits for memory.
#include "decay.h"

namespace dlrm {
namespace seq {
namespace decay {
namespace {

// LP: d rounded up to 32, 64 or 128.  LP / 4 threads a row, ROWS rows at once, N of them a thread.
template <int LP>
__global__ __launch_bounds__(LP == 32 ? 64 : 256) void k_decay_step(const Walk a, float *state) {
    constexpr int THREADS = LP == 32 ? 64 : 256, COLS = LP / 4, ROWS = THREADS / COLS, N = LP / ROWS;
    constexpr int HEADS = 4;  // whose sums over rows are joined at once
    __shared__ __attribute__((aligned(16))) float ks[LP], qs[HEADS][LP], sums[HEADS][ROWS][LP];
    const int64_t id = blockIdx.x;
    const int64_t b = id / a.Hkv;
    const int kvh = static_cast<int>(id % a.Hkv), tid = threadIdx.x;
    const int col = tid % COLS * 4, row = tid / COLS;
    float *S = state + id * a.d * a.d;
    const bool in = col < a.d;

    floatx4 s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = floatx4{0.f, 0.f, 0.f, 0.f};
        if (in && i * ROWS + row < a.d) s[i] = *(const DLRM_GLOBAL floatx4 *)(S + (i * ROWS + row) * a.d + col);
    }
    floatx4 v = {0.f, 0.f, 0.f, 0.f};
    if (in) {
        const u32x2 x = *(const DLRM_GLOBAL u32x2 *)(a.z.p + b * a.z.row + kvh * a.z.head + col);
        v = floatx4{bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y)};
    }
    for (int i = tid; i < LP; i += THREADS)
        ks[i] = i < a.d ? bf16_lo(a.y.p[b * a.y.row + kvh * a.y.head + i]) : 0.f;
    float g = a.g[b * a.g_row + kvh];
    g = g > 0.f ? 0.f : g < kLeast ? kLeast : g;
    const float f = expf(g);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float k = ks[i * ROWS + row];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = fmaf(f, s[i][e], k * v[e]);
        if (in && i * ROWS + row < a.d) *(DLRM_GLOBAL floatx4 *)(S + (i * ROWS + row) * a.d + col) = s[i];
    }
    const int h0 = kvh * a.group;
    for (int h = 0; h < a.group; h += HEADS) {
        const int n = min(HEADS, a.group - h);
        if (h) __syncthreads();  // the sums before have been read
        for (int i = tid; i < n * LP; i += THREADS) {
            const int c = i % LP;
            qs[i / LP][c] = c < a.d ? bf16_lo(a.x.p[b * a.x.row + (h0 + h + i / LP) * a.x.head + c]) : 0.f;
        }
        __syncthreads();
        for (int j = 0; j < n; ++j) {
            floatx4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float q = qs[j][i * ROWS + row];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = fmaf(q, s[i][e], o[e]);
            }
            *reinterpret_cast<floatx4 *>(&sums[j][row][col]) = o;
        }
        __syncthreads();
        for (int i = tid; i < n * (LP / 2); i += THREADS) {
            const int j = i / (LP / 2), c = i % (LP / 2) * 2;
            if (c >= a.d) continue;
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) x += sums[j][r][c], y += sums[j][r][c + 1];
            *(DLRM_GLOBAL uint32_t *)(a.out + (b * a.Hq + h0 + h + j) * a.d + c) = pack_bf16(x * a.scale, y * a.scale);
        }
    }
}

template <int LP>
int launch(const Walk &a, float *state, hipStream_t stream) {
    DLRM_LAUNCH("seq_decay_step", k_decay_step<LP>, dim3(static_cast<uint32_t>(a.B * a.Hkv)), dim3(LP == 32 ? 64 : 256), 0, stream, a, state);
    return launch_status();
}

}  // namespace
}  // namespace decay
}  // namespace seq
}  // namespace dlrm

extern "C" int dlrm_seq_decay_step(const dlrm_seq_decay *desc, float *state, uint16_t *o, dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq::decay;
    Walk a;
    const int rc = check(desc, false, &a);
    if (rc != DLRM_OK) return rc;
    if (desc->N != desc->B) return DLRM_ERR_INVALID_ARG;
    if (static_cast<int64_t>(a.B) * a.Hkv >= (1 << 24)) return DLRM_ERR_UNSUPPORTED;
    if (a.B == 0) return DLRM_OK;
    if (!o || !state || !aligned(o, 16) || !aligned(state, 16)) return DLRM_ERR_INVALID_ARG;
    a.out = o;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    if (a.d <= 32) return launch<32>(a, state, stream);
    if (a.d <= 64) return launch<64>(a, state, stream);
    return launch<128>(a, state, stream);
}
