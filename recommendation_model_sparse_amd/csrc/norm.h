// Shared by the residual norm's and dropout's kernels (dlrm_seq.h): the counter-based generator, typed
// loads and stores, sums over a row's lanes.
#pragma once

#include "common.h"
#include "dlrm_seq.h"

namespace dlrm {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

struct Drop {
    uint32_t limit;  // an element whose 16 bits are below it is dropped; 0: no dropout
    float scale;
    uint32_t k0, k1;
    uint64_t offset;
    const uint64_t *offset_dev;
};

inline bool drop_of(const dlrm_dropout_spec *s, Drop *out) {
    *out = Drop{};
    if (!s || s->p == 0.f) return true;
    if (!(s->p > 0.f && s->p <= 1.f) || !aligned(s->offset_dev, 8)) return false;
    out->limit = static_cast<uint32_t>(static_cast<double>(s->p) * 65536.0 + 0.5);
    out->scale = out->limit == 65536 ? 0.f : 65536.f / static_cast<float>(65536 - out->limit);
    out->k0 = static_cast<uint32_t>(s->seed), out->k1 = static_cast<uint32_t>(s->seed >> 32);
    out->offset = s->offset, out->offset_dev = s->offset_dev;
    return true;
}

// Philox4x32-10: the multipliers and key increments of the paper; the counter's upper half is 0.
// 16 bits an element rather than 32: each number then serves twice as many, and its 20 wide
// multiplications (a quarter of the plain rate) stay below what the memory allows.
__device__ __forceinline__ u32x4 philox(uint64_t counter, uint32_t k0, uint32_t k1) {
    uint32_t x0 = static_cast<uint32_t>(counter), x1 = static_cast<uint32_t>(counter >> 32), x2 = 0, x3 = 0;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = static_cast<uint64_t>(x0) * 0xD2511F53u, b = static_cast<uint64_t>(x2) * 0xCD9E8D57u;
        x0 = static_cast<uint32_t>(b >> 32) ^ x1 ^ k0, x1 = static_cast<uint32_t>(b);
        x2 = static_cast<uint32_t>(a >> 32) ^ x3 ^ k1, x3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
    }
    return u32x4{x0, x1, x2, x3};
}

// Bit e: element 8 * group + e is kept.
__device__ __forceinline__ uint32_t keep_bits(const Drop &d, uint64_t offset, uint64_t group) {
    const u32x4 r = philox(offset + group, d.k0, d.k1);
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bits |= ((r[i] & 0xffffu) >= d.limit ? 1u : 0u) << (2 * i);
        bits |= ((r[i] >> 16) >= d.limit ? 2u : 0u) << (2 * i);
    }
    return bits;
}

__device__ __forceinline__ uint64_t base_offset(const Drop &d) { return d.offset + (d.offset_dev ? *d.offset_dev : 0); }

// Workgroups of 256 in a launch, which holds fewer than 2^32 work-items; more rows are several launches.
constexpr int64_t kMostBlocks = (int64_t(1) << 24) - 1;

// ---------------------------------------------------------------- typed loads and stores

struct F32 {};
struct BF16 {};
struct F8 {};

template <typename T>
struct Size { static constexpr int bytes = 4; };
template <>
struct Size<BF16> { static constexpr int bytes = 2; };
template <>
struct Size<F8> { static constexpr int bytes = 1; };

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// V (8 or 1) consecutive elements from index e on; 8 of them are aligned to 16 bytes.
template <typename T, int V>
__device__ __forceinline__ void load(const void *p, int64_t e, float *x) {
    const char *at = static_cast<const char *>(p) + e * Size<T>::bytes;
    if constexpr (V == 1) {
        if constexpr (Size<T>::bytes == 4) x[0] = *(const DLRM_GLOBAL float *)at;
        else x[0] = __uint_as_float(static_cast<uint32_t>(*(const DLRM_GLOBAL uint16_t *)at) << 16);
    } else if constexpr (Size<T>::bytes == 4) {
        uint32_t w[8];
        gload_words<8>(at, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
        uint32_t w[4];
        gload_words<4>(at, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
    }
}

template <typename T, int V>
__device__ __forceinline__ void store(void *p, int64_t e, const float *x) {
    char *at = static_cast<char *>(p) + e * Size<T>::bytes;
    if constexpr (V == 1) {
        if constexpr (Size<T>::bytes == 4) *(DLRM_GLOBAL float *)at = x[0];
        else if constexpr (Size<T>::bytes == 2) *(DLRM_GLOBAL uint16_t *)at = static_cast<uint16_t>(pack2(x[0], 0.f));
        else *(DLRM_GLOBAL uint8_t *)at = static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[0], 0, false));
    } else if constexpr (Size<T>::bytes == 4) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
        gstore_words<8>(at, w);
    } else if constexpr (Size<T>::bytes == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1]);
        gstore_words<4>(at, w);
    } else {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
            w[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], v, true));
        }
        gstore_words<2>(at, w);
    }
}

// x rounded to T and back: what a reader of the stored value sees.
template <typename T>
__device__ __forceinline__ float rounded(float x) {
    if constexpr (Size<T>::bytes == 2) return bf16_lo(pack2(x, 0.f));
    return x;
}

// Orders one wavefront's LDS writes before its lanes' reads of each other's.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------- sums over a row's lanes

struct Add { __device__ float operator()(float a, float b) const { return a + b; } };
struct Max { __device__ float operator()(float a, float b) const { return fmaxf(a, b); } };

// L lanes (16, 32, 64, or a workgroup of 256, then through `part`) hold one row.
template <int L, typename Op>
__device__ __forceinline__ float over_row(float x, float *part, Op op) {
#pragma unroll
    for (int i = 1; i < (L < 64 ? L : 64); i <<= 1) x = op(x, __shfl_xor(x, i));
    if constexpr (L == 256) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
        __syncthreads();
        x = op(op(part[0], part[1]), op(part[2], part[3]));
    }
    return x;
}

// The dropout factors of a row's elements.  Rows of whole groups of 8 (V = 8): one number a piece.
// Others (V = 1, piece i of a wavefront's lane at column base + LW i + lane): the groups that the
// lanes of a row segment cover are numbered through, each lane makes N / 8 of them, and their bits go
// through LDS, a byte a group; a number an element would be eight times the work.
template <int LW, int N, int V>
struct Keep {
    static constexpr int GROUPS = LW * N / 8 + 1;
    typedef uint8_t Bytes[256 / LW][GROUPS + 7];
    const uint8_t *mine;
    int64_t first;  // element of the segment's first column

    // Before the row's factors are asked for (V = 1): columns [0, cols) of the segment are in use.
    __device__ __forceinline__ void row(const Drop &d, uint64_t offset, Bytes &bytes, int64_t e0, int cols) {
        const int sub = threadIdx.x % LW, seg = threadIdx.x / LW;
        const int last = static_cast<int>(((e0 & 7) + cols - 1) >> 3);
        wave_lds_sync();
#pragma unroll
        for (int k = 0; k < N / 8; ++k)
            if (LW * k + sub <= last) bytes[seg][LW * k + sub] = static_cast<uint8_t>(keep_bits(d, offset, (e0 >> 3) + LW * k + sub));
        if (last >= LW * N / 8 && sub == 0) bytes[seg][LW * N / 8] = static_cast<uint8_t>(keep_bits(d, offset, (e0 >> 3) + LW * N / 8));
        wave_lds_sync();
        mine = bytes[seg], first = e0;
    }
    __device__ __forceinline__ void get(const Drop &d, uint64_t offset, int64_t e, float *m) const {
        if constexpr (V == 8) {
            const uint32_t bits = keep_bits(d, offset, static_cast<uint64_t>(e) >> 3);
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = bits >> j & 1 ? d.scale : 0.f;
        } else {
            m[0] = mine[(e >> 3) - (first >> 3)] >> (e & 7) & 1 ? d.scale : 0.f;
        }
    }
};

// Column of piece i: rows of 8-element groups go round the row's lanes; others give each wavefront a
// run of its own, for Keep.
template <int L, int N, int V>
__device__ __forceinline__ int column(int i) {
    const int lane = threadIdx.x % L;
    if constexpr (V == 8 || L < 256) return (lane + L * i) * V;
    return (lane >> 6) * 64 * N + 64 * i + (lane & 63);
}

// A kept element times the scale, a dropped one 0 (not its value times 0: that may be NaN).
__device__ __forceinline__ float drop_one(float x, float m) { return m == 0.f ? 0.f : x * m; }

inline bool is_float(int32_t t) { return t == DLRM_F32 || t == DLRM_BF16; }

inline int widest(int D) { return D % 8 == 0 ? 16384 : 4096; }

// The lanes of a row and the pieces of a lane, by the width: rows of whole 8-element groups (16-byte
// accesses), others element by element.  A wavefront holds a row while it fits 32 values a lane.
// Forward + backward in us for 2^24 bf16 elements with dropout, and with about twice the lanes:
//   width 64: 65 / 112, 128: 46 / 63, 256: 46 / 62, 512: 46 / 46, 1024: 46 / 55, 2048: 49 / 45 (but 1032:
//   58 / 62 and 4096: 48 / 48);  odd: 100: 86 / 153, 479: 89 / 393
// with half the lanes: 256: 48, 1024: 50, 2048: 77, 4096: 65; odd 479: 90.
// Odd widths up to 2048 take 8 pieces a lane (1500: 162, 2001: 130), as 16 leave half the lanes without
// any and cost 423 and 332.
template <typename A, typename B, typename C, typename P>
void by_width(const P &p) {
    const int D = p.D;
    if (D % 8 == 0) {
        if (D <= 128) P::template run<A, B, C, 16, 1, 8>(p);
        else if (D <= 256) P::template run<A, B, C, 32, 1, 8>(p);
        else if (D <= 512) P::template run<A, B, C, 64, 1, 8>(p);
        else if (D <= 1024) P::template run<A, B, C, 64, 2, 8>(p);
        else if (D <= 2048) P::template run<A, B, C, 64, 4, 8>(p);
        else if (D <= 8192) P::template run<A, B, C, 256, 4, 8>(p);
        else P::template run<A, B, C, 256, 8, 8>(p);
    } else {
        if (D <= 128) P::template run<A, B, C, 16, 8, 1>(p);
        else if (D <= 512) P::template run<A, B, C, 64, 8, 1>(p);
        else if (D <= 1024) P::template run<A, B, C, 64, 16, 1>(p);
        else if (D <= 2048) P::template run<A, B, C, 256, 8, 1>(p);
        else P::template run<A, B, C, 256, 16, 1>(p);
    }
}

}  // namespace
}  // namespace dlrm
