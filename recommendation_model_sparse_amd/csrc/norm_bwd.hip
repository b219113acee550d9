// The RMS norm with the residual's addition and dropout, backward (dlrm_seq.h).
//
//   dh = ds + rstd (dy w - hat mean(dy w hat)), hat = s rstd;  dx = m dh;  dw = sum dy hat
//
// Bound by reading and writing each row once, as the forward.  Measured, for its cases: 150000 x 128 53
// us, 5.8 TB/s; 16384 x 479 fp32 36 us, 4.4; dw's sum over the workgroups 6 us.  Odd widths past 2048 are far
// from that (4195 x 3999 bf16: 212 us): a workgroup holds one row, and 256 registers a lane leave one
// wavefront a SIMD; a bound on the registers made it 294.
#include "norm.h"

namespace dlrm {
namespace {

// A workgroup walks rows blockIdx.x, + gridDim.x, ...: its lanes keep the columns they own, and sum
// dw over the rows in registers.  partial: [gridDim.x][D].
template <typename G, typename R, typename X, int L, int N, int V, bool DROP>
__global__ __launch_bounds__(256) void k_add_rmsnorm_bwd(const void *dy, const void *ds, const void *s, const float *w,
                                                         const float *rstd, Drop drop, int64_t M, int D, void *dx, void *dres,
                                                         float *partial) {
    constexpr int ROWS = 256 / L, LW = L < 64 ? L : 64;
    __shared__ float part[4];
    __shared__ typename Keep<LW, V == 1 ? N : 8, V>::Bytes bytes;
    __shared__ float join[ROWS > 1 ? 256 * N * V : 1];
    const int lane = threadIdx.x % L, sub = threadIdx.x / L;
    const uint64_t offset = DROP ? base_offset(drop) : 0;
    float wv[N * V], dw[N * V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = column<L, N, V>(i);
#pragma unroll
        for (int j = 0; j < V; ++j) wv[i * V + j] = dw[i * V + j] = 0.f;
        if (c < D) load<F32, V>(w, c, wv + i * V);
    }
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + sub; row < M; row += static_cast<int64_t>(gridDim.x) * ROWS) {
        const float inv = rstd[row];
        Keep<LW, V == 1 ? N : 8, V> keep;
        if constexpr (DROP && V == 1) {
            const int c0 = L == 256 ? lane / 64 * 64 * N : 0;
            if (c0 < D) keep.row(drop, offset, bytes, row * D + c0, min(D - c0, LW * N));
        }
        float g[N * V], hat[N * V], dot = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = column<L, N, V>(i);
#pragma unroll
            for (int j = 0; j < V; ++j) g[i * V + j] = hat[i * V + j] = 0.f;
            if (c >= D) continue;
            load<G, V>(dy, row * D + c, g + i * V);
            load<R, V>(s, row * D + c, hat + i * V);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int k = i * V + j;
                hat[k] *= inv;
                dw[k] = fmaf(g[k], hat[k], dw[k]);
                g[k] *= wv[k];
                dot = fmaf(g[k], hat[k], dot);
            }
        }
        const float mean = over_row<L>(dot, part, Add()) / static_cast<float>(D);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = column<L, N, V>(i);
            if (c >= D) continue;
            const int64_t e = row * D + c;
            float d[V];
            if (ds) load<R, V>(ds, e, d);
            else {
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = fmaf(inv, g[i * V + j] - hat[i * V + j] * mean, d[j]);
            if (dres) store<R, V>(dres, e, d);
            if constexpr (DROP) {
                float m[V];
                keep.get(drop, offset, e, m);
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = drop_one(d[j], m[j]);
            }
            store<X, V>(dx, e, d);
        }
    }
    if constexpr (ROWS > 1) {  // the rows that ran side by side, in order
#pragma unroll
        for (int k = 0; k < N * V; ++k) join[k * 256 + threadIdx.x] = dw[k];
        __syncthreads();
        if (sub != 0) return;
#pragma unroll
        for (int k = 0; k < N * V; ++k) {
            float x = 0.f;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) x += join[k * 256 + r * L + lane];
            dw[k] = x;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = column<L, N, V>(i);
        if (c < D) store<F32, V>(partial, static_cast<int64_t>(blockIdx.x) * D + c, dw + i * V);
    }
}

// dw[c] = sum over the workgroups' partial sums: 16 columns by 64 runs of rows, then the runs in order.
__global__ __launch_bounds__(1024) void k_rmsnorm_dw(const float *partial, int rows, int D, float *dw) {
    __shared__ float part[64][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, c = blockIdx.x * 16 + tx;
    float x = 0.f;
    if (c < D) {
#pragma unroll 16
        for (int r = ty; r < rows; r += 64) x += partial[static_cast<int64_t>(r) * D + c];
    }
    part[ty][tx] = x;
    __syncthreads();
    if (ty < 8) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y += part[8 * ty + i][tx];
        part[8 * ty][tx] = y;
    }
    __syncthreads();
    if (ty == 0 && c < D) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) y += part[8 * i][tx];
        dw[c] = y;
    }
}

struct Bwd {
    const void *dy, *ds, *s;
    const float *w, *rstd;
    Drop drop;
    int64_t M;
    int D;
    void *dx, *dres;
    float *partial, *dw;
    int blocks;
    hipStream_t stream;

    template <typename A, typename B, typename C, int L, int N, int V>
    static void run(const Bwd &);
};

template <typename G, typename R, typename X, int L, int N, int V>
void Bwd::run(const Bwd &b) {
    const dim3 grid(static_cast<uint32_t>(b.blocks));
    if (b.drop.limit)
        DLRM_LAUNCH("add_rmsnorm_bwd", (k_add_rmsnorm_bwd<G, R, X, L, N, V, true>), grid, dim3(256), 0, b.stream, b.dy, b.ds, b.s,
                    b.w, b.rstd, b.drop, b.M, b.D, b.dx, b.dres, b.partial);
    else
        DLRM_LAUNCH("add_rmsnorm_bwd", (k_add_rmsnorm_bwd<G, R, X, L, N, V, false>), grid, dim3(256), 0, b.stream, b.dy, b.ds, b.s,
                    b.w, b.rstd, b.drop, b.M, b.D, b.dx, b.dres, b.partial);
}

int rows_at_once(int D) { return D <= 128 ? 16 : D <= 256 && D % 8 == 0 ? 8 : D <= (D % 8 == 0 ? 2048 : 1024) ? 4 : 1; }

// Workgroups of the backward: four a CU, fewer where the rows or the table of their dw sums (8 MB)
// do not ask for them.
int bwd_blocks(int64_t M, int D) {
    const int64_t r = rows_at_once(D), want = (M + r - 1) / r;
    int64_t most = (int64_t(1) << 21) / D;
    most = most < 256 ? 256 : most > 1024 ? 1024 : most;
    return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

}  // namespace
}  // namespace dlrm

extern "C" size_t dlrm_add_rmsnorm_bwd_workspace_size(int64_t M, int32_t D) {
    using namespace dlrm;
    if (M < 0 || D < 1 || D > widest(D) || M >= (int64_t(1) << 31)) return 0;
    return static_cast<size_t>(bwd_blocks(M, D)) * D * 4 + 256;
}

extern "C" int dlrm_add_rmsnorm_bwd(const void *dy, int32_t dy_dtype, const void *ds, const void *s, int32_t res_dtype,
                                    const float *w, const float *rstd, const dlrm_dropout_spec *spec, int64_t M, int32_t D,
                                    void *dx, int32_t x_dtype, void *dresidual, float *dw, void *workspace,
                                    size_t workspace_bytes, dlrm_stream_t stream_) {
    using namespace dlrm;
    Bwd b{};
    if (M < 0 || D < 1 || !is_float(dy_dtype) || !is_float(res_dtype) || !is_float(x_dtype) || !drop_of(spec, &b.drop))
        return DLRM_ERR_INVALID_ARG;
    if (D > widest(D) || M >= (int64_t(1) << 31)) return DLRM_ERR_UNSUPPORTED;
    if (!w || !dw || !aligned(w, 16) || !aligned(dw, 4) || !aligned(dy, 16) || !aligned(ds, 16) || !aligned(s, 16) ||
        !aligned(rstd, 4) || !aligned(dx, 16) || !aligned(dresidual, 16))
        return DLRM_ERR_INVALID_ARG;
    if (M > 0 && (!dy || !s || !rstd || !dx)) return DLRM_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < dlrm_add_rmsnorm_bwd_workspace_size(M, D))
        return DLRM_ERR_WORKSPACE;
    b.dy = dy, b.ds = ds, b.s = s, b.w = w, b.rstd = rstd, b.M = M, b.D = D, b.dx = dx, b.dres = dresidual;
    b.partial = static_cast<float *>(workspace), b.dw = dw, b.blocks = bwd_blocks(M, D);
    b.stream = reinterpret_cast<hipStream_t>(stream_);
    const auto by_x = [&](auto G, auto R) {
        using GT = decltype(G);
        using RT = decltype(R);
        if (x_dtype == DLRM_F32) by_width<GT, RT, F32>(b);
        else by_width<GT, RT, BF16>(b);
    };
    if (dy_dtype == DLRM_F32 && res_dtype == DLRM_F32) by_x(F32(), F32());
    else if (dy_dtype == DLRM_F32) by_x(F32(), BF16());
    else if (res_dtype == DLRM_F32) by_x(BF16(), F32());
    else by_x(BF16(), BF16());
    DLRM_LAUNCH("rmsnorm_dw", k_rmsnorm_dw, dim3((D + 15) / 16), dim3(1024), 0, b.stream, static_cast<const float *>(b.partial),
                b.blocks, D, dw);
    return launch_status();
}
