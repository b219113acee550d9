// The RMS norm with the residual's addition and dropout, forward, and dropout alone (dlrm_seq.h).
//
//   s = residual + m x;  rstd = (mean s^2 + eps)^-1/2;  y = s rstd w
//
// Bound by reading and writing each row once: a row stays in the registers of 16, 32, 64 or 256
// lanes between its sum and its use, and the dropout factors m are made where they are applied.
// Measured: 150000 rows of 128, x and y bf16, s fp32, dropout: 42 us, 5.4 TB/s; 16384 of 1024 bf16 to 8
// bits: 24 us, 4.9; 16384 of 479 fp32, element by element: 26 us, 4.8; dropout alone on 16384 x 1024 fp32:
// 23 us, 5.7 (a large copy: 5.15).
#include <algorithm>

#include "norm.h"

namespace dlrm {
namespace {

// One row by L lanes, each with N pieces of V elements (columns: column<L, N, V>).
template <typename X, typename R, typename Y, int L, int N, int V, bool DROP>
__global__ __launch_bounds__(256) void k_add_rmsnorm_fwd(const void *x, const void *res, const float *w, float eps, Drop drop,
                                                         int64_t row0, int64_t M, int D, void *s, void *y, float *y_scale,
                                                         float *rstd) {
    constexpr int LW = L < 64 ? L : 64;
    __shared__ float part[4];
    __shared__ typename Keep<LW, V == 1 ? N : 8, V>::Bytes bytes;
    const int lane = threadIdx.x % L;
    const int64_t row = row0 + static_cast<int64_t>(blockIdx.x) * (256 / L) + threadIdx.x / L;
    if (row >= M) return;  // L == 256: the whole workgroup
    const uint64_t offset = DROP ? base_offset(drop) : 0;
    Keep<LW, V == 1 ? N : 8, V> keep;
    if constexpr (DROP && V == 1) {
        const int c0 = L == 256 ? lane / 64 * 64 * N : 0;
        if (c0 < D) keep.row(drop, offset, bytes, row * D + c0, min(D - c0, LW * N));
    }
    float h[N * V], sq = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = column<L, N, V>(i);
#pragma unroll
        for (int j = 0; j < V; ++j) h[i * V + j] = 0.f;
        if (c >= D) continue;
        const int64_t e = row * D + c;
        float a[V], r[V];
        load<X, V>(x, e, a);
        if (res) load<R, V>(res, e, r);
        else {
#pragma unroll
            for (int j = 0; j < V; ++j) r[j] = 0.f;
        }
        if constexpr (DROP) {
            float m[V];
            keep.get(drop, offset, e, m);
#pragma unroll
            for (int j = 0; j < V; ++j) a[j] = drop_one(a[j], m[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            a[j] = rounded<R>(r[j] + a[j]);
            h[i * V + j] = a[j];
            sq = fmaf(a[j], a[j], sq);
        }
        if (s) store<R, V>(s, e, a);
    }
    sq = over_row<L>(sq, part, Add());
    const float inv = 1.f / sqrtf(sq / static_cast<float>(D) + eps);
    if (rstd && lane == 0) rstd[row] = inv;
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = column<L, N, V>(i);
        if (c >= D) continue;
        float g[V];
        load<F32, V>(w, c, g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            h[i * V + j] *= inv * g[j];
            if constexpr (Size<Y>::bytes == 1) most = fmaxf(most, fabsf(h[i * V + j]));
        }
        if constexpr (Size<Y>::bytes != 1) store<Y, V>(y, row * D + c, h + i * V);
    }
    if constexpr (Size<Y>::bytes == 1) {
        most = over_row<L>(most, part, Max());
        // divided by the scale as it is stored, which a product with 448 / most misses by an 8-bit step here and
        // there (12 of 2^24).  One reciprocal a row and a correction by the remainder give the rounded quotient
        // (Markstein, 1990) while nothing leaves the normal numbers (what is smaller than the scale by 2^12 is 0
        // in 8 bits either way); a division an element took 27.3 us where this takes 24.3 (16384 of 1024).  A
        // scale below the normal numbers is kept above 0, and its quotients within range.
        const float scale = most == 0.f ? 1.f : fmaxf(most / 448.f, 0x1p-149f), inverse = 1.f / scale;
        const bool normal = scale > 0x1p-90f && scale < 0x1p100f;
        if (lane == 0) y_scale[row] = scale;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = column<L, N, V>(i);
            if (c >= D) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float q = h[i * V + j] * inverse;
                if (normal) {
                    q = fmaf(fmaf(-q, scale, h[i * V + j]), inverse, q);
                } else {
                    q = h[i * V + j] / scale;
                    q = fabsf(q) > 448.f ? copysignf(448.f, q) : q;
                }
                h[i * V + j] = q;
            }
            store<F8, V>(y, row * D + c, h + i * V);
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_dropout(const void *x, int64_t group0, int64_t n, Drop drop, void *y) {
    const int64_t group = group0 + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, e = group * 8;
    if (e >= n) return;
    const uint32_t bits = keep_bits(drop, base_offset(drop), static_cast<uint64_t>(group));
    if (e + 8 <= n) {
        float v[8];
        load<T, 8>(x, e, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = bits >> j & 1 ? v[j] * drop.scale : 0.f;
        store<T, 8>(y, e, v);
    } else {
        for (int j = 0; e + j < n; ++j) {
            float v;
            load<T, 1>(x, e + j, &v);
            v = bits >> j & 1 ? v * drop.scale : 0.f;
            store<T, 1>(y, e + j, &v);
        }
    }
}

struct Fwd {
    const void *x, *res;
    const float *w;
    float eps;
    Drop drop;
    int64_t M;
    int D;
    void *s, *y;
    float *y_scale, *rstd;
    hipStream_t stream;

    template <typename A, typename B, typename C, int L, int N, int V>
    static void run(const Fwd &);
};

template <typename X, typename R, typename Y, int L, int N, int V>
void Fwd::run(const Fwd &f) {
    constexpr int64_t most = kMostBlocks * (256 / L);
    for (int64_t row0 = 0; row0 < f.M; row0 += most) {
        const dim3 grid(static_cast<uint32_t>((std::min(f.M - row0, most) + 256 / L - 1) / (256 / L)));
        if (f.drop.limit)
            DLRM_LAUNCH("add_rmsnorm_fwd", (k_add_rmsnorm_fwd<X, R, Y, L, N, V, true>), grid, dim3(256), 0, f.stream, f.x, f.res,
                        f.w, f.eps, f.drop, row0, f.M, f.D, f.s, f.y, f.y_scale, f.rstd);
        else
            DLRM_LAUNCH("add_rmsnorm_fwd", (k_add_rmsnorm_fwd<X, R, Y, L, N, V, false>), grid, dim3(256), 0, f.stream, f.x, f.res,
                        f.w, f.eps, f.drop, row0, f.M, f.D, f.s, f.y, f.y_scale, f.rstd);
    }
}

}  // namespace
}  // namespace dlrm

extern "C" int dlrm_dropout(const void *x, int32_t dtype, int64_t n, const dlrm_dropout_spec *spec, void *y,
                            dlrm_stream_t stream_) {
    using namespace dlrm;
    Drop drop;
    if (n < 0 || !is_float(dtype) || !spec || !drop_of(spec, &drop)) return DLRM_ERR_INVALID_ARG;
    if (n >= (int64_t(1) << 40)) return DLRM_ERR_UNSUPPORTED;
    if (n == 0) return DLRM_OK;
    if (!x || !y || !aligned(x, 16) || !aligned(y, 16)) return DLRM_ERR_INVALID_ARG;
    if (!drop.limit) drop.scale = 1.f;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    const int64_t groups = (n + 7) / 8, most = kMostBlocks * 256;
    for (int64_t g = 0; g < groups; g += most) {
        const dim3 grid(static_cast<uint32_t>((std::min(groups - g, most) + 255) / 256));
        if (dtype == DLRM_F32)
            DLRM_LAUNCH("dropout", k_dropout<F32>, grid, dim3(256), 0, stream, x, g, n, drop, y);
        else
            DLRM_LAUNCH("dropout", k_dropout<BF16>, grid, dim3(256), 0, stream, x, g, n, drop, y);
    }
    return launch_status();
}

extern "C" int dlrm_add_rmsnorm_fwd(const void *x, int32_t x_dtype, const void *residual, int32_t res_dtype, const float *w,
                                    float eps, const dlrm_dropout_spec *spec, int64_t M, int32_t D, void *s, void *y,
                                    int32_t y_dtype, float *y_scale, float *rstd, dlrm_stream_t stream_) {
    using namespace dlrm;
    Fwd f{};
    if (M < 0 || D < 1 || !is_float(x_dtype) || !is_float(res_dtype) || !(is_float(y_dtype) || y_dtype == DLRM_F8_E4M3) ||
        !(eps >= 0.f) || !drop_of(spec, &f.drop))
        return DLRM_ERR_INVALID_ARG;
    if (D > widest(D) || M >= (int64_t(1) << 31)) return DLRM_ERR_UNSUPPORTED;
    if (!w || !aligned(w, 16) || !aligned(x, 16) || !aligned(residual, 16) || !aligned(s, 16) || !aligned(y, 16) ||
        !aligned(rstd, 4) || !aligned(y_scale, 4))
        return DLRM_ERR_INVALID_ARG;
    if (M > 0 && (!x || !y || (y_dtype == DLRM_F8_E4M3 && !y_scale))) return DLRM_ERR_INVALID_ARG;
    if (M == 0) return DLRM_OK;
    f.x = x, f.res = residual, f.w = w, f.eps = eps, f.M = M, f.D = D, f.s = s, f.y = y, f.y_scale = y_scale, f.rstd = rstd;
    f.stream = reinterpret_cast<hipStream_t>(stream_);
    const auto by_y = [&](auto X, auto R) {
        using XT = decltype(X);
        using RT = decltype(R);
        if (y_dtype == DLRM_F32) by_width<XT, RT, F32>(f);
        else if (y_dtype == DLRM_BF16) by_width<XT, RT, BF16>(f);
        else by_width<XT, RT, F8>(f);
    };
    if (x_dtype == DLRM_F32 && res_dtype == DLRM_F32) by_y(F32(), F32());
    else if (x_dtype == DLRM_F32) by_y(F32(), BF16());
    else if (res_dtype == DLRM_F32) by_y(BF16(), F32());
    else by_y(BF16(), BF16());
    return launch_status();
}
