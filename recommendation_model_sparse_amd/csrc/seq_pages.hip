// The paged cache of user histories (dlrm_seq_pages.h): the tables of a visit, and rows to their slots.
//
// A visit is a handful of sums over users, then independent reads and writes.  Users are taken 1024 a
// workgroup, one a thread: how many pages each gives back and wants, and the sums before it; then all pages of
// the 1024, and all new events, are spread over the threads, each of which finds its user in the sums.  Up to 1024
// users and 16384 events are one launch of one workgroup, which is bound by its chain of reads (a launch
// and five of them); more take four launches, as pages that are taken may have come back in another workgroup, or three if nobody leaves.
// Measured: 256 users of up to 512 events, one new one each, 7.8 us; 20000 with a million new events, 29 us: 4.5, 6.7, 6.9, 11.4.
#include "seq.h"

namespace dlrm {
namespace seq {
namespace {

constexpr int kUsers = 1024;        // a workgroup's, one a thread
constexpr int kFewEvents = 16384;   // that one workgroup places
constexpr int kRun = 256;           // events that a wavefront places

struct Visit {
    int32_t *table, *lengths, *free_list, *free_count;
    int64_t row, pages, N;
    const void *off;
    const uint8_t *leave;
    int64_t *slots;
    int32_t *refused;
    int32_t idx32, B, width, shift;
    // workspace: per 1024 users what they give back and want; the stack's top before and after the pages that come
    // back, pages taken; the events of each user before its new ones, -1: refused
    int64_t *sums, *tops;
    int32_t *base;
};

struct User {
    int64_t n;
    int held, have, gone, want;  // events and pages held (after leaving); pages given back; pages wanted
    bool wide;
};

__device__ __forceinline__ User user_of(const Visit &a, int b) {
    User u = {};
    if (b >= a.B) return u;
    const int o0 = offset_at(a, a.off, b, a.N), o1 = offset_at(a, a.off, b + 1, a.N);
    const int most = a.width << a.shift, held = min(max(a.lengths[b], 0), most);
    const bool leaves = a.leave && a.leave[b];
    const int page = 1 << a.shift, have = (held + page - 1) >> a.shift;
    u.n = max(o1 - o0, 0);
    u.gone = leaves ? have : 0;
    u.held = leaves ? 0 : held, u.have = leaves ? 0 : have;
    u.wide = u.held + u.n <= most;
    u.want = u.wide ? static_cast<int>((u.held + u.n + page - 1) >> a.shift) - u.have : 0;
    return u;
}

struct Scan {
    int64_t wave[kUsers / 64];
};

// The sum over the workgroup's threads up to this one, and over all.
__device__ __forceinline__ int64_t scan(Scan &lds, int64_t x, int64_t *all) {
    const int lane = threadIdx.x & 63, w = static_cast<int>(wave_id());
    int64_t s = x;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
        const int64_t up = __shfl_up(s, i);
        if (lane >= i) s += up;
    }
    __syncthreads();
    if (lane == 63) lds.wave[w] = s;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int v = 0; v < kUsers / 64; ++v) {
        if (v == w) s += total;
        total += lds.wave[v];
    }
    *all = total;
    return s;
}

// The last thread whose sum before it is at most k: sums[i] is that of thread i, ending in one of all.
__device__ __forceinline__ int owner(const int64_t *sums, int64_t k) {
    int lo = 0, hi = kUsers;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= k) lo = mid;
        else hi = mid;
    }
    return lo;
}

// What the workgroups before this one have of entry `which` of sums, and all of them in *all; each wavefront by itself.
__device__ __forceinline__ int64_t before(const Visit &a, int which, int64_t *all) {
    const int blocks = (a.B + kUsers - 1) / kUsers;
    int64_t mine = 0, total = 0;
    for (int i = static_cast<int>(__lane_id()); i < blocks; i += 64) {
        const int64_t x = a.sums[2 * i + which];
        total += x;
        if (i < static_cast<int>(blockIdx.x)) mine += x;
    }
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) mine += __shfl_xor(mine, i), total += __shfl_xor(total, i);
    *all = total;
    return mine;
}

struct Lds {
    Scan scan;
    int64_t sums[kUsers], start[kUsers];
    int32_t have[kUsers];
};

// Pages of users who leave go onto the stack from `top` on, in order.
__device__ __forceinline__ void give_back(const Visit &a, Lds &lds, const User &u, int64_t top) {
    const int t = static_cast<int>(threadIdx.x), b0 = static_cast<int>(blockIdx.x) * kUsers;
    int64_t all;
    const int64_t upto = scan(lds.scan, u.gone, &all);
    lds.sums[t] = upto - u.gone;
    __syncthreads();
    for (int64_t k = t; k < all; k += kUsers) {
        const int i = owner(lds.sums, k);
        int32_t *entry = a.table + (b0 + i) * a.row + (k - lds.sums[i]);
        if (top + k < a.pages) a.free_list[top + k] = *entry;
        *entry = -1;
    }
    if (u.gone) a.lengths[b0 + t] = 0;
}

// Pages from the stack's top for those whom it has them for; `first`: wanted in the workgroups before.  Returns
// whether it has them for this thread's user; in all, *taken pages, and users *refused.
__device__ __forceinline__ bool take(const Visit &a, Lds &lds, const User &u, int64_t top, int64_t first, int64_t *taken, int64_t *refused) {
    const int t = static_cast<int>(threadIdx.x), b0 = static_cast<int>(blockIdx.x) * kUsers;
    int64_t all;
    const int64_t upto = scan(lds.scan, u.want, &all);  // its barriers are behind the reads of lds.sums
    const bool fits = u.wide && (u.want == 0 || first + upto <= top);
    // who is refused wants pages that are not there, or none: those who get some are the first ones who want any
    lds.sums[t] = upto - u.want, lds.have[t] = fits ? u.have : -1;
    int64_t both;
    scan(lds.scan, (fits ? static_cast<int64_t>(u.want) << 20 : 0) + (b0 + t < a.B && !fits ? 1 : 0), &both);
    *taken = both >> 20, *refused = both & ((1 << 20) - 1);
    for (int64_t k = t; k < *taken; k += kUsers) {
        const int i = owner(lds.sums, k);
        a.table[(b0 + i) * a.row + lds.have[i] + (k - lds.sums[i])] = a.free_list[top - 1 - first - k];
    }
    if (b0 + t < a.B && fits && u.n) a.lengths[b0 + t] = static_cast<int32_t>(u.held + u.n);
    return fits;
}

__device__ __forceinline__ int64_t slot_of(const Visit &a, int b, int held, int64_t i) {
    const int64_t p = held + i;
    return (static_cast<int64_t>(a.table[b * a.row + (p >> a.shift)]) << a.shift) + (p & ((1 << a.shift) - 1));
}

__device__ __forceinline__ int64_t top_of(const Visit &a) {
    return min(static_cast<int64_t>(max(*a.free_count, 0)), a.pages);
}

// Few users: all of it.  PLACE: the events' slots too.
template <bool PLACE>
__global__ __launch_bounds__(kUsers) void k_pages_visit(const Visit a) {
    __shared__ Lds lds;
    const int t = static_cast<int>(threadIdx.x);
    const User u = user_of(a, t);
    const int64_t top0 = top_of(a);
    int64_t gone, taken, refused;
    scan(lds.scan, u.gone, &gone);
    if (gone) give_back(a, lds, u, top0);
    const int64_t top = min(top0 + gone, a.pages);
    __syncthreads();  // the stack as it is now
    const bool fits = take(a, lds, u, top, 0, &taken, &refused);
    if (t == 0) *a.free_count = static_cast<int32_t>(top - taken), *a.refused = static_cast<int32_t>(refused);
    if constexpr (PLACE) {
        // sums over the users' events; their rows begin at the first offset
        int64_t events;
        const int64_t upto = scan(lds.scan, u.n, &events);
        lds.sums[t] = upto - u.n, lds.have[t] = fits ? u.held : -1;
        lds.start[t] = t < a.B ? offset_at(a, a.off, t, a.N) : 0;
        __syncthreads();
        for (int64_t k = t; k < events; k += kUsers) {
            const int i = owner(lds.sums, k), held = lds.have[i];
            const int64_t at = k - lds.sums[i], row = lds.start[i] + at;
            if (row < a.N) a.slots[row] = held < 0 ? -1 : slot_of(a, i, held, at);
        }
    } else {
        if (t < a.B) a.base[t] = fits ? u.held : -1;
    }
}

__global__ __launch_bounds__(kUsers) void k_pages_count(const Visit a) {
    __shared__ Scan lds;
    const User u = user_of(a, static_cast<int>(blockIdx.x * kUsers + threadIdx.x));
    int64_t gone, want;
    scan(lds, u.gone, &gone);
    scan(lds, u.want, &want);
    if (threadIdx.x != 0) return;
    a.sums[2 * blockIdx.x] = gone, a.sums[2 * blockIdx.x + 1] = want;
    if (blockIdx.x == 0) a.tops[0] = top_of(a), a.tops[1] = 0, *a.refused = 0;
}

__global__ __launch_bounds__(kUsers) void k_pages_give_back(const Visit a) {
    __shared__ Lds lds;
    const User u = user_of(a, static_cast<int>(blockIdx.x * kUsers + threadIdx.x));
    int64_t all;
    const int64_t first = before(a, 0, &all);
    if (all) give_back(a, lds, u, a.tops[0] + first);
}

__global__ __launch_bounds__(kUsers) void k_pages_take(const Visit a) {
    __shared__ Lds lds;
    const int b = static_cast<int>(blockIdx.x * kUsers + threadIdx.x);
    Visit now = a;
    now.leave = nullptr;  // they are empty by now
    const User u = user_of(now, b);
    int64_t gone, want, taken, refused;
    before(a, 0, &gone);
    const int64_t first = before(a, 1, &want);
    const bool fits = take(a, lds, u, min(a.tops[0] + gone, a.pages), first, &taken, &refused);
    if (b < a.B) a.base[b] = fits ? u.held : -1;
    if (threadIdx.x != 0) return;
    if (refused) atomicAdd(a.refused, static_cast<int32_t>(refused));
    if (taken) atomicAdd(reinterpret_cast<unsigned long long *>(a.tops + 1), static_cast<unsigned long long>(taken));
}

// The events' slots, kRun of a user's a wavefront; `many`: the stack's count too, which the launches before leave.
__global__ __launch_bounds__(256) void k_pages_place(const Visit a, uint32_t runs, bool many) {
    if (many && blockIdx.x == 0 && threadIdx.x == 0) {
        int64_t gone = 0;
        for (int i = 0; i < (a.B + kUsers - 1) / kUsers; ++i) gone += a.sums[2 * i];
        *a.free_count = static_cast<int32_t>(min(a.tops[0] + gone, a.pages) - a.tops[1]);
    }
    const uint32_t run = blockIdx.x * 4 + wave_id();
    if (run >= runs) return;
    const int b = find_sequence(a, a.off, a.N, static_cast<int>(run), kRun);
    const int64_t o0 = offset_at(a, a.off, b, a.N), n = offset_at(a, a.off, b + 1, a.N) - o0;
    const int64_t first = (static_cast<int64_t>(run) - (o0 / kRun + b)) * kRun;
    if (first < 0 || first >= n) return;
    const int held = a.base[b];
#pragma unroll
    for (int i = 0; i < kRun; i += 64) {
        const int64_t at = first + i + (threadIdx.x & 63);
        if (at < n) a.slots[o0 + at] = held < 0 ? -1 : slot_of(a, b, held, at);
    }
}

struct Rows {
    uint16_t *p;
    int64_t row, head;
};

// 16 bytes of a key's and a value's row a thread.  2900 rows of 2 heads of 128: 4.4 us; fewer are bound by the launch.
__global__ __launch_bounds__(256) void k_pages_write(Rows k, Rows v, Rows k_pool, Rows v_pool, const int64_t *slots, int64_t N, int64_t rows,
                                                     uint32_t per_row, uint32_t per_head) {
    const uint64_t all = static_cast<uint64_t>(N) * per_row;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < all; i += gridDim.x * 256ull) {
        const uint64_t n = all >> 32 ? i / per_row : static_cast<uint32_t>(i) / per_row;
        const uint32_t c = static_cast<uint32_t>(i - n * per_row), h = c / per_head, e = 8 * (c - h * per_head);
        const int64_t s = slots[n];
        if (s < 0 || s >= rows) continue;
        const int64_t r = static_cast<int64_t>(n);
        const u32x4 x = *(const DLRM_GLOBAL u32x4 *)(k.p + r * k.row + h * k.head + e);
        const u32x4 y = *(const DLRM_GLOBAL u32x4 *)(v.p + r * v.row + h * v.head + e);
        *(DLRM_GLOBAL u32x4 *)(k_pool.p + s * k_pool.row + h * k_pool.head + e) = x;
        *(DLRM_GLOBAL u32x4 *)(v_pool.p + s * v_pool.row + h * v_pool.head + e) = y;
    }
}

size_t sums_bytes(int64_t B) { return (16 * static_cast<size_t>((B + kUsers - 1) / kUsers + 1) + 255) / 256 * 256; }

}  // namespace
}  // namespace seq
}  // namespace dlrm

extern "C" size_t dlrm_seq_pages_update_workspace_size(int64_t B, int64_t N) {
    if (B < 0 || B >= (1 << 20) || N < 0 || N >= (int64_t(1) << 31)) return 0;
    return 256 + dlrm::seq::sums_bytes(B) + 4 * static_cast<size_t>(B);
}

extern "C" int dlrm_seq_pages_update(const dlrm_seq_pages *p, const void *offsets, int32_t index_type, int64_t N, const uint8_t *leave,
                                     int64_t *slots, int32_t *refused, void *workspace, size_t workspace_bytes, dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq;
    if (!p || p->B < 0 || N < 0 || p->pages < 1 || p->width < 0 || p->table_row < p->width) return DLRM_ERR_INVALID_ARG;
    if (index_type != DLRM_INDEX_I64 && index_type != DLRM_INDEX_I32) return DLRM_ERR_INVALID_ARG;
    if (p->page < 8 || p->page > 4096 || (p->page & (p->page - 1)) != 0) return DLRM_ERR_UNSUPPORTED;
    if (p->B >= (1 << 20) || N >= (int64_t(1) << 31) || p->pages >= (int64_t(1) << 31) / p->page ||
        static_cast<int64_t>(p->width) * p->page >= (int64_t(1) << 30))
        return DLRM_ERR_UNSUPPORTED;
    const uintptr_t ib = index_type == DLRM_INDEX_I32 ? 4 : 8;
    if (!p->free_list || !p->free_count || !refused || !aligned(p->free_list, 4) || !aligned(p->free_count, 4) || !aligned(refused, 4))
        return DLRM_ERR_INVALID_ARG;
    if (p->B > 0 && (!p->lengths || (!p->table && p->width > 0) || !offsets || !aligned(p->lengths, 4) || !aligned(p->table, 4) ||
                     !aligned(offsets, ib)))
        return DLRM_ERR_INVALID_ARG;
    if (N > 0 && (!slots || !aligned(slots, 8))) return DLRM_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < dlrm_seq_pages_update_workspace_size(p->B, N)) return DLRM_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    Visit a = {};
    a.table = p->table, a.lengths = p->lengths, a.free_list = p->free_list, a.free_count = p->free_count;
    a.row = p->table_row, a.pages = p->pages, a.N = N;
    a.off = offsets, a.leave = leave, a.slots = slots, a.refused = refused;
    a.idx32 = index_type == DLRM_INDEX_I32, a.B = static_cast<int32_t>(p->B), a.width = p->width, a.shift = __builtin_ctz(p->page);
    a.tops = reinterpret_cast<int64_t *>(ws);
    a.sums = reinterpret_cast<int64_t *>(ws + 256);
    a.base = reinterpret_cast<int32_t *>(ws + 256 + sums_bytes(p->B));
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    const bool many = p->B > kUsers, place = many || N > kFewEvents;
    if (!many) {
        if (place) DLRM_LAUNCH("seq_pages_visit", (k_pages_visit<false>), dim3(1), dim3(kUsers), 0, stream, a);
        else DLRM_LAUNCH("seq_pages_visit", (k_pages_visit<true>), dim3(1), dim3(kUsers), 0, stream, a);
    } else {
        const dim3 blocks(static_cast<uint32_t>((p->B + kUsers - 1) / kUsers));
        DLRM_LAUNCH("seq_pages_count", k_pages_count, blocks, dim3(kUsers), 0, stream, a);
        if (leave) DLRM_LAUNCH("seq_pages_give_back", k_pages_give_back, blocks, dim3(kUsers), 0, stream, a);
        DLRM_LAUNCH("seq_pages_take", k_pages_take, blocks, dim3(kUsers), 0, stream, a);
    }
    if (place && p->B > 0) {
        const uint32_t runs = static_cast<uint32_t>(slot_count(N, p->B, kRun));
        DLRM_LAUNCH("seq_pages_place", k_pages_place, dim3((runs + 3) / 4), dim3(256), 0, stream, a, runs, many);
    }
    return launch_status();
}

extern "C" int dlrm_seq_pages_write(const uint16_t *k, int64_t k_row, int64_t k_head, const uint16_t *v, int64_t v_row, int64_t v_head,
                                    int64_t N, int32_t H, int32_t d, const int64_t *slots, uint16_t *k_pool, int64_t k_pool_row,
                                    int64_t k_pool_head, uint16_t *v_pool, int64_t v_pool_row, int64_t v_pool_head, int64_t rows,
                                    dlrm_stream_t stream_) {
    using namespace dlrm;
    using namespace dlrm::seq;
    if (N < 0 || rows < 0 || H < 1 || d < 1) return DLRM_ERR_INVALID_ARG;
    if (d % 8 != 0 || static_cast<int64_t>(H) * d > (1 << 20) || N >= (int64_t(1) << 31)) return DLRM_ERR_UNSUPPORTED;
    const int64_t strides[8] = {k_row, k_head, v_row, v_head, k_pool_row, k_pool_head, v_pool_row, v_pool_head};
    for (int64_t s : strides)
        if (s % 8 != 0 || s < d) return DLRM_ERR_INVALID_ARG;
    if (N == 0 || rows == 0) return DLRM_OK;
    const void *all[4] = {k, v, k_pool, v_pool};
    for (const void *x : all)
        if (!x || !aligned(x, 16)) return DLRM_ERR_INVALID_ARG;
    if (!slots || !aligned(slots, 8)) return DLRM_ERR_INVALID_ARG;
    const uint32_t per_head = d / 8, per_row = H * per_head;
    const uint64_t blocks = (static_cast<uint64_t>(N) * per_row + 255) / 256;
    const uint32_t grid = static_cast<uint32_t>(blocks < (1u << 20) ? blocks : 1u << 20);
    DLRM_LAUNCH("seq_pages_write", k_pages_write, dim3(grid), dim3(256), 0, reinterpret_cast<hipStream_t>(stream_),
                (Rows{const_cast<uint16_t *>(k), k_row, k_head}), (Rows{const_cast<uint16_t *>(v), v_row, v_head}), (Rows{k_pool, k_pool_row, k_pool_head}),
                (Rows{v_pool, v_pool_row, v_pool_head}), slots, N, rows, per_row, per_head);
    return launch_status();
}
