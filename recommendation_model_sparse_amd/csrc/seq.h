// Shared by the attention kernels over jagged sequences (dlrm_seq.h): arguments, the map from
// workgroups to tiles of sequences, LDS tiles and matrix-core fragments.
#pragma once

#include "common.h"
#include "dlrm_seq.h"
#include "dlrm_seq_pages.h"

namespace dlrm {
namespace seq {

constexpr int kBK = 64;  // rows of a staged tile (keys; queries in the backward over keys)
constexpr int kQT = 64;  // queries of a workgroup
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_inff();
// Above this a maximum or log-sum of the logits is rounded by more than 2^-4, and exp(z - m) is
// taken from the difference itself instead of from one fused multiply-add in base 2: a row whose
// every visible bias is -1e9, or the type's lowest value, still has z - m = 0.
constexpr float kHuge = 0x1p20f;

struct Args {
    const uint16_t *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    const void *q_off, *kv_begin, *kv_end;
    int64_t Nq, Nkv;
    int32_t B, Hq, Hkv, group, d;
    int32_t idx32;
    int32_t window, sinks;
    float scale;  // of <q, k>
    const float *bias;
    int32_t buckets;   // 0 without a bias
    int32_t last;      // first distance of the last bucket: from there on the bias is one value
    int32_t bounds[DLRM_SEQ_MAX_BUCKETS];
};

// Checks the description and fills Args (host).  `paged`: the keys are in pages, and have no offsets.
int check_attn(const dlrm_seq_attn *a, bool need_q_offsets, Args *out, bool paged = false);

// Which rows of a pool hold the events of a sequence (dlrm_seq_pages.h).
struct Pages {
    const int32_t *table, *lengths;
    int64_t row;  // of the table
    int32_t width, shift, last;  // pages of a sequence, log2 of a page's events, the pool's last page
};

// Checks the tables against the description and fills Pages (host).
int check_pages(const dlrm_seq_attn *a, const dlrm_seq_pages *p, Pages *out);

__device__ __forceinline__ int paged_length(const Pages &pg, int b) { return min(max(pg.lengths[b], 0), pg.width << pg.shift); }

// The pool's row of event x; `table`: the sequence's.  What is no page counts as the last one.
__device__ __forceinline__ int paged_row(const Pages &pg, const int32_t *table, int x) {
    const uint32_t page = min(static_cast<uint32_t>(table[x >> pg.shift]), static_cast<uint32_t>(pg.last));
    return static_cast<int>((page << pg.shift) + (x & ((1 << pg.shift) - 1)));
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

union Frag {  // eight bf16 values: one lane's share of an MFMA operand
    uint32_t w[4];
    u32x4 q;
    s16x4 h[2];
    bf16x8 b;
};

// Two fp32 -> two bf16, round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Entry i of an offset array, brought into [0, limit] (limit < 2^31; what is negative is limit).
// `a`: Args, or another kernel's with its idx32.
template <typename A>
__device__ __forceinline__ int offset_at(const A &a, const void *p, int64_t i, int64_t limit) {
    if (a.idx32) {
        const uint32_t x = static_cast<const uint32_t *>(p)[i];
        return static_cast<int>(min(x, static_cast<uint32_t>(limit)));
    }
    const uint64_t x = static_cast<const uint64_t *>(p)[i];
    return static_cast<int>(x < static_cast<uint64_t>(limit) ? static_cast<uint32_t>(x) : static_cast<uint32_t>(limit));
}

// Tiles of T rows over B jagged sequences without a table of them: sequence b owns the slots from
// off[b] / T + b on.  It needs ceil(len / T) <= off[b+1] / T - off[b] / T + 1 of them, so no two
// sequences meet; rows / T + B slots cover all, and those a sequence does not need end at once.
__host__ __device__ __forceinline__ int64_t slot_count(int64_t rows, int64_t B, int T) { return rows / T + B; }

// The sequence that owns a slot, by one wavefront, as every probe waits for memory: 64 probes at
// once, twice for up to 4096 sequences.
template <typename A>
__device__ __forceinline__ int find_sequence(const A &a, const void *off, int64_t limit, int slot, int T) {
    int lo = 0, n = a.B;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int at = static_cast<int>(__lane_id()) * step;
        bool below = false;
        if (at < n) below = offset_at(a, off, lo + at, limit) / static_cast<uint32_t>(T) + lo + at <= static_cast<uint32_t>(slot);
        const int c = max(1, __popcll(__ballot(below)));  // none: offsets that are not in order
        lo += (c - 1) * step;
        n = min(step, n - (c - 1) * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

struct Span {  // one sequence
    int64_t q0, k0;  // first rows
    int qlen, klen;
    int shift;       // position of query 0
};

__device__ __forceinline__ Span span_of(const Args &a, int b) {
    const int q0 = offset_at(a, a.q_off, b, a.Nq), q1 = offset_at(a, a.q_off, b + 1, a.Nq);
    const int k0 = offset_at(a, a.kv_begin, b, a.Nkv), k1 = offset_at(a, a.kv_end, b, a.Nkv);
    Span s;
    s.q0 = q0, s.k0 = k0;
    s.qlen = max(q1 - q0, 0), s.klen = max(k1 - k0, 0);
    s.shift = s.klen - s.qlen;
    return s;
}

__device__ __forceinline__ Span span_of(const Args &a, const Pages &pg, int b) {
    const int q0 = offset_at(a, a.q_off, b, a.Nq), q1 = offset_at(a, a.q_off, b + 1, a.Nq);
    Span s;
    s.q0 = q0, s.k0 = 0;
    s.qlen = max(q1 - q0, 0), s.klen = paged_length(pg, b);
    s.shift = s.klen - s.qlen;
    return s;
}

// ---------------------------------------------------------------- LDS tiles
//
// A tile holds 64 rows of LP elements (LP = 32, 64 or 128: the head's width rounded up), 8 or 16
// elements apart: the rows that one read instruction touches (8 of 16 bytes, or 4 of 32 in the
// transposing read) lie in different banks, and every address is a lane's base plus a constant
// (swapping 16-byte chunks instead cost about 25 registers of addresses).

template <int LP>
constexpr int kPitch = LP == 64 ? 72 : LP + 16;

// A lane's place in a tile for read_row: row `row`, columns from 8 * half on.
template <int LP>
__device__ __forceinline__ int row_base(int row, int half) {
    return row * kPitch<LP> + 8 * half;
}

// One lane's 8 bf16 at step i (16 columns a step).
__device__ __forceinline__ void read_row(Frag &f, const uint16_t *at, int i) {
    f.q = *reinterpret_cast<const u32x4 *>(at + 16 * i);
}

// Transposed operand of v_mfma_f32_32x32x16_bf16 from a row-major tile: lane l gets column
// col0 + (l & 31) of the rows row0 + 4 * (l >> 5) + {0..3} and those 8 further on.  That is the
// order in which the accumulator of the product before holds its rows, so that its values are this
// product's other operand as they stand.  Within 16 lanes ds_read_b64_tr_b16 takes 4 rows of 16
// columns, lane i reading 4 columns of row i / 4, and gives lane i column i of the 4 rows.
template <int LP>
__device__ __forceinline__ int column_base(int lane) {
    const int i = lane & 15;
    return (4 * (lane >> 5) + (i >> 2)) * kPitch<LP> + (lane & 16) + 4 * (i & 3);
}

template <int LP>
__device__ __forceinline__ void read_columns(Frag &f, const uint16_t *at, int row0, int col0) {
    typedef __attribute__((address_space(3))) s16x4 *lds_t;
#pragma unroll
    for (int g = 0; g < 2; ++g)
        f.h[g] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(at + (row0 + 8 * g) * kPitch<LP> + col0));
}

// 64 rows of a [rows][d] bf16 matrix on their way to LDS, through registers: `load` issues the
// reads for a tile (rows outside [first, end), but for those below `sinks`, are zeros, as are
// columns from d on), `store` writes it.  The next tile is not read ahead: its 16 to 32 registers a
// matrix cost a wavefront a SIMD, which hides more (heads of 128: 361 -> 318 us for the backward's
// first kernel; of 64: no difference).
template <int LP, int THREADS, int BK = kBK>
struct Stage {
    static constexpr int CH = LP / 8;
    static constexpr int N = BK * CH / THREADS;  // 16-byte pieces a thread
    static constexpr int R = THREADS / CH;        // rows that are read at once
    u32x4 r[N];
    int row, lds;
    uint32_t at;
    bool col;

    __device__ __forceinline__ Stage(int64_t stride, int d) {
        const int c = threadIdx.x % CH;
        row = threadIdx.x / CH;
        lds = row * kPitch<LP> + 8 * c;
        at = static_cast<uint32_t>(row) * static_cast<uint32_t>(stride) * 2 + 16 * c;
        col = 8 * c < d;
    }
    __device__ __forceinline__ void load(const uint16_t *base, int64_t stride, int d, int row0, int first, int end, int sinks) {
        const char *p = reinterpret_cast<const char *>(base + row0 * stride);
        const int64_t step = R * stride * 2;
        if (d == LP && row0 >= first && row0 + BK <= end) {
#pragma unroll
            for (int i = 0; i < N; ++i, p += step) r[i] = *(const DLRM_GLOBAL u32x4 *)(p + at);
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i, p += step) {
            const int x = row0 + i * R + row;
            r[i] = u32x4{0, 0, 0, 0};
            if (col && x < end && (x >= first || x < sinks)) r[i] = *(const DLRM_GLOBAL u32x4 *)(p + at);
        }
    }
    // The rows of a thread's pieces in a pool of pages, and the pieces from there.  Nothing branches, as each branch
    // waits: a row past the end reads the last one, and what is not wanted is left out on its way to the tile.
    __device__ __forceinline__ void paged_rows(int (&at)[N], const Pages &pg, const int32_t *table, int row0, int end) const {
#pragma unroll
        for (int i = 0; i < N; ++i) at[i] = paged_row(pg, table, min(row0 + i * R + row, end - 1));
    }
    __device__ __forceinline__ void load_rows(const uint16_t *base, int64_t stride, const int (&at)[N]) {
        const int c = col ? 8 * (threadIdx.x % CH) : 0;
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = *(const DLRM_GLOBAL u32x4 *)(base + at[i] * stride + c);
    }
    __device__ __forceinline__ void store_rows(uint16_t *tile, int row0, int first, int end, int sinks) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int x = row0 + i * R + row;
            if (!(col && x < end && (x >= first || x < sinks))) r[i] = u32x4{0, 0, 0, 0};
        }
        store(tile);
    }
    __device__ __forceinline__ void store(uint16_t *tile) const {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4 *>(tile + lds + i * R * kPitch<LP>) = r[i];
    }
};

// Two bf16 with infinities and NaN replaced by zeros.
__device__ __forceinline__ uint32_t only_finite(uint32_t x) {
    const uint32_t lo = (x & 0x7f80u) == 0x7f80u ? 0u : x & 0xffffu;
    const uint32_t hi = (x & 0x7f800000u) == 0x7f800000u ? 0u : x & 0xffff0000u;
    return lo | hi;
}

// Orders one wavefront's LDS writes before its lanes' reads of each other's.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The maximum (sum) of a value over the two lanes l and l ^ 32.
__device__ __forceinline__ float max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ---------------------------------------------------------------- bias by distance

// The bucket of distance n >= 0: the last t with bounds[t] <= n.
template <typename Bounds>
__device__ __forceinline__ int bucket_of(const Bounds *bounds, int buckets, int n) {
    int lo = 0, hi = buckets;  // bounds[lo] <= n < bounds[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (bounds[mid] <= n) lo = mid;
        else hi = mid;
    }
    return lo;
}

// What is added to the logits at distance n: the bias, or -infinity where the distance is not visible.
// `past_window`: the window is left to the caller, who knows which keys are first ones.
template <typename Bounds, typename Bias>
__device__ __forceinline__ float bias_at(const Args &a, const Bounds *bounds, const Bias *bias, int n, bool past_window, int *bucket) {
    const int t = n > 0 && a.buckets ? bucket_of(bounds, a.buckets, n) : 0;
    *bucket = t;
    if (n < 0 || (a.window && n >= a.window && !past_window)) return -kInf;
    return a.buckets ? bias[t] : 0.f;
}

// A workgroup looks the biases of the distances [-kPad, NEAR) up once, as far as its tiles need them;
// a tile's distances are a run of them.  (A table for each tile took 960 of its 6190 cycles in
// the forward, heads of 128: every search is a chain of LDS reads.)  Tiles further out have a table of their own, unless the bias is
// one value there.
constexpr int kPad = 128;

}  // namespace seq
}  // namespace dlrm
