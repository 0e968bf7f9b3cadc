// pages.hip - pages of the paged cache: rows of a block table that grow and
// shrink, rows that share another one's pages, copies of pages, and the move of
// an accepted path's keys and values.
//
// A pool's state is refs[pages], how many table entries name a page (0: free),
// and held[b], how many pages row b of the table holds, in its first entries.
// Free pages are taken lowest first, in the order of the rows and their entries,
// so results do not depend on the order in which threads run.
#include "forward.hpp"

namespace dspark {

constexpr int kPoolThreads = 1024;
constexpr int kPoolWaves = kPoolThreads / kWave;
constexpr int kRefRows = 16;  // entries of refs that a thread looks at together
constexpr int kPoolWords = kRefRows * kPoolWaves + 4;  // of LDS for scans
constexpr int kMoveThreads = 128;
constexpr int kCopyThreads = 256;

// Inclusive sum over the workgroup; `all` gets the total.
__device__ __forceinline__ int pool_scan(int x, int *lds, int &all) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int in = wave_incl_scan(x, lane);
    __syncthreads();
    if (lane == kWave - 1) lds[wave] = in;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kPoolWaves; ++w) {
        before += w < wave ? lds[w] : 0;
        sum += lds[w];
    }
    all = sum;
    return before + in;
}

__device__ __forceinline__ void release(int32_t *refs, int pages, int page) {
    if (page >= 0 && page < pages) atomicSub(refs + page, 1);
}
__device__ __forceinline__ int clamped(int x, int lo, int hi) {
    return x < lo ? lo : (x > hi ? hi : x);
}

// Takes the lowest free pages from `from` (a multiple of what is looked at together) on:
// take(rank, page) is called for ranks 0 .. need - 1 as far as there are free pages.
// Returns how many there were; `from` is left where the next search goes on.
// Entries of refs are read past the vector cache, which the atomics on them do not go
// through, 16 rows of 1024 at a time: a page's rank is a count of bits.
template <typename Take>
__device__ __forceinline__ int take_free(int32_t *refs, int pages, int &from, int need, int *lds,
                                         Take take) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    int found = 0;
    while (found < need && from < pages) {
        int32_t r[kRefRows];
#pragma unroll
        for (int i = 0; i < kRefRows; ++i) {
            const int page = from + i * kPoolThreads + threadIdx.x;
            r[i] = page < pages ? __hip_atomic_load(refs + page, __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT)
                                : 1;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRefRows; ++i) {
            const uint64_t free = __ballot(r[i] == 0);
            if (lane == 0) lds[i * kPoolWaves + wave] = __popcll(free);
        }
        __syncthreads();
        // the first 256 threads hold the counts of the waves' rows in the pages' order
        static_assert(kRefRows * kPoolWaves == 4 * kWave, "four waves scan the counts");
        int count = 0, in = 0;
        if (wave < 4) {
            count = lds[threadIdx.x];
            in = wave_incl_scan(count, lane);
            if (lane == kWave - 1) lds[kRefRows * kPoolWaves + wave] = in;
        }
        __syncthreads();
        const int *sums = lds + kRefRows * kPoolWaves;
        if (wave < 4) {
            for (int w = 0; w < wave; ++w) in += sums[w];
            lds[threadIdx.x] = in - count;
        }
        const int all = sums[0] + sums[1] + sums[2] + sums[3];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRefRows; ++i) {
            const uint64_t free = __ballot(r[i] == 0);
            const int rank = found + lds[i * kPoolWaves + wave] +
                             __popcll(free & ((1ull << lane) - 1));
            if (r[i] == 0 && rank < need) {
                const int page = from + i * kPoolThreads + threadIdx.x;
                refs[page] = 1;
                take(rank, page);
            }
        }
        found += all;
        if (found <= need) from += kPoolThreads * kRefRows;
    }
    __syncthreads();
    return found < need ? found : need;
}

// For each x[u] the last index b[u] of the non-decreasing before[kPoolThreads] in LDS
// with before[b[u]] <= x[u], step by step for all of them.
template <int kN>
__device__ __forceinline__ void owners(const int *before, const int (&x)[kN], int (&b)[kN]) {
#pragma unroll
    for (int u = 0; u < kN; ++u) b[u] = 0;
#pragma unroll
    for (int step = kPoolThreads / 2; step > 0; step >>= 1) {
        int y[kN];
#pragma unroll
        for (int u = 0; u < kN; ++u) y[u] = before[b[u] + step];
#pragma unroll
        for (int u = 0; u < kN; ++u) b[u] += y[u] <= x[u] ? step : 0;
    }
}
__device__ __forceinline__ int owner(const int *before, int x) {
    int xs[1] = {x}, b[1];
    owners(before, xs, b);
    return b[0];
}

// One workgroup, 1024 rows at a time: first every row's pages past its length are
// released, then the rows that need more take theirs. Both work on the entries of
// all rows laid end to end, so one long row costs no more than many short ones. A
// chain of dependent reads: 2.4 us for 8 to 1000 rows that keep what they hold, 3.8 to
// 7.5 where each gives a page back and 6.2 to 8.3 where each takes one and free pages are
// among the first 16384; 12000 releases 19 us, by the rate of one compute unit's atomics
// (more workgroups would need a second launch before pages are taken). The search for
// free pages begins at page 0 in every call that takes any, 4 us for every 16384 pages
// that it passes: 30 us in all behind 100 000 taken pages, 250 behind a million.
__global__ __launch_bounds__(kPoolThreads) void resize_pages_kernel(PoolParams p) {
    __shared__ int before_s[kPoolThreads], held_s[kPoolThreads], lds[kPoolWords];
    auto rows_from = [&](int b0, int &held, int &want) {
        const int b = b0 + threadIdx.x;
        held = want = 0;
        if (b >= p.R) return;
        held = clamped(p.held[b], 0, p.width);
        const int64_t len = p.lens[b] < 0 ? 0 : p.lens[b];
        const int64_t n = (len + p.page - 1) / p.page;
        want = n > p.width ? -1 : (int)n;  // more than a row can hold: not served
    };
    int held = 0, want = 0;
    for (int b0 = 0; b0 < p.R; b0 += kPoolThreads) {
        int all;
        rows_from(b0, held, want);
        const int less = want >= 0 && held > want ? held - want : 0;
        const int in = pool_scan(less, lds, all);
        before_s[threadIdx.x] = in - less;
        held_s[threadIdx.x] = want;
        __syncthreads();
        constexpr int kAhead = 8;  // entries on their way a thread
        for (int i0 = threadIdx.x; i0 < all; i0 += kAhead * kPoolThreads) {
            int32_t *e[kAhead];
            int page[kAhead], i[kAhead], b[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                i[u] = i0 + u * kPoolThreads < all ? i0 + u * kPoolThreads : i0;
            owners(before_s, i, b);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                e[u] = p.table + (int64_t)(b0 + b[u]) * p.width + held_s[b[u]] +
                       (i[u] - before_s[b[u]]);
                page[u] = *e[u];
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (i0 + u * kPoolThreads >= all) break;
                release(p.refs, p.pages, page[u]);
                *e[u] = -1;
            }
        }
        if (less > 0) p.held[b0 + threadIdx.x] = want;
        if (b0 + (int)threadIdx.x < p.R) p.granted[b0 + threadIdx.x] = want >= 0;
        __syncthreads();
    }
    __syncthreads();
    int from = 0;
    bool short_of = false;
    for (int b0 = 0; b0 < p.R; b0 += kPoolThreads) {
        int all;
        if (p.R > kPoolThreads) rows_from(b0, held, want);
        const int more = want > held ? want - held : 0;
        const int in = pool_scan(more, lds, all);
        if (all == 0) continue;
        before_s[threadIdx.x] = in - more;
        held_s[threadIdx.x] = held;
        __syncthreads();
        auto entry = [&](int rank) {
            const int b = owner(before_s, rank);
            return p.table + (int64_t)(b0 + b) * p.width + held_s[b] + (rank - before_s[b]);
        };
        int got = 0;
        if (!short_of)
            got = take_free(p.refs, p.pages, from, all, lds,
                            [&](int rank, int page) { *entry(rank) = page; });
        // from the first row on that cannot have all of its pages none gets any
        const bool served = in <= got;
        if (more > 0 && served) p.held[b0 + threadIdx.x] = want;
        if (more > 0 && !served) p.granted[b0 + threadIdx.x] = 0;
        if (got < all) {  // that row gives back what it got
            const int first = before_s[owner(before_s, got)];
            for (int rank = first + threadIdx.x; rank < got; rank += kPoolThreads) {
                int32_t *e = entry(rank);
                release(p.refs, p.pages, *e);
                *e = -1;
            }
            short_of = true;
        }
        __syncthreads();
    }
}

// Positions of row s that fork i takes: at most what the row holds.
__device__ __forceinline__ int64_t fork_length(const PoolParams &p, int s) {
    const int64_t most = (int64_t)clamped(p.held[s], 0, p.width) * p.page;
    const int64_t len = p.lens[s] < 0 ? 0 : p.lens[s];
    return len < most ? len : most;
}

// Fork i by `threads` threads: the target's old pages go, the source's full pages and
// the fresh one come. The source keeps its own hold on what is shared, so no page
// looks free in between, whatever the order.
__device__ __forceinline__ int fork_row(const PoolParams &p, int i, int tid, int threads) {
    const int s = p.src[i], d = p.dst[i], fresh = p.copy_dst[i];
    const int old = clamped(p.held[d], 0, p.width);
    const int full = (int)(fork_length(p, s) / p.page), now = full + (fresh >= 0);
    const int32_t *in = p.table + (int64_t)s * p.width;
    int32_t *out = p.table + (int64_t)d * p.width;
    const int last = now > old ? now : old;
    for (int e = tid; e < last; e += threads) {
        const int page = e < full ? in[e] : (e < now ? fresh : -1);
        if (e < full && page >= 0 && page < p.pages) atomicAdd(p.refs + page, 1);
        if (e < old) release(p.refs, p.pages, out[e]);
        out[e] = page;
    }
    return now;
}

// One workgroup: which forks are granted, and a fresh page for each that ends
// inside a page. kAll: and the forks themselves, a wave each. A chain of six dependent
// reads, 6.6 us for three forks and 7.5 for 17 (3 more on cold caches), and the
// comparison of every target with all rows named, 0.05 us a fork: 64 forks take 9.5 us,
// 224 17, 512 33 and 1024 77, and every 1024 are compared with all. Free pages are
// searched for as by resize_pages_kernel.
template <bool kAll>
__global__ __launch_bounds__(kPoolThreads) void fork_plan_kernel(PoolParams p) {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    __shared__ i32x4 src_s[kPoolThreads / 4], dst_s[kPoolThreads / 4];
    __shared__ int fresh_s[kPoolThreads], lds[kPoolWords];
    int from = 0;
    bool short_of = false;
    for (int i0 = 0; i0 < p.n; i0 += kPoolThreads) {
        const int i = i0 + threadIdx.x;
        int s = -1, d = -1;
        if (i < p.n) {
            s = p.src[i];
            d = p.dst[i];
        }
        bool ok = s >= 0 && s < p.R && d >= 0 && d < p.R;
        // a row is the target of one fork, and not read by any
        for (int k0 = 0; k0 < p.n; k0 += kPoolThreads) {
            const int k = k0 + threadIdx.x;
            __syncthreads();
            reinterpret_cast<int *>(src_s)[threadIdx.x] = k < p.n ? p.src[k] : -1;
            reinterpret_cast<int *>(dst_s)[threadIdx.x] = k < p.n ? p.dst[k] : -1;
            __syncthreads();
            int m = p.n - k0 < kPoolThreads ? p.n - k0 : kPoolThreads;
            if (!__any(i < p.n)) m = 0;
#pragma unroll 4
            for (int u = 0; u < m; u += 4) {
                const i32x4 a = src_s[u / 4], z = dst_s[u / 4];
#pragma unroll
                for (int v = 0; v < 4; ++v)  // -1 past the last entry is no row
                    ok &= d != a[v] && (d != z[v] || k0 + u + v >= i);
            }
        }
        int part = -1, rest = 0;
        if (ok) {
            const int64_t len = fork_length(p, s);
            const int full = (int)(len / p.page);
            rest = (int)(len - (int64_t)full * p.page);
            if (rest > 0) part = p.table[(int64_t)s * p.width + full];
        }
        const int need = rest > 0;
        int all;
        const int in = pool_scan(need, lds, all);
        fresh_s[threadIdx.x] = -1;
        __syncthreads();
        int got = 0;
        if (!short_of && all > 0)
            got = take_free(p.refs, p.pages, from, all, lds,
                            [&](int rank, int page) { fresh_s[rank] = page; });
        __syncthreads();
        if (need && in > got) ok = false;
        if (i < p.n) {
            const int fresh = ok && need ? fresh_s[in - 1] : -1;
            const bool copied = fresh >= 0 && part >= 0 && part < p.pages;
            p.copy_src[i] = copied ? part : -1;
            p.copy_dst[i] = fresh;
            p.copy_slots[i] = copied ? rest : 0;
            p.granted[i] = ok;
        }
        short_of |= got < all;
    }
    if constexpr (kAll) {
        __syncthreads();
        const int lane = threadIdx.x & (kWave - 1);
        for (int i = threadIdx.x / kWave; i < p.n; i += kPoolWaves) {
            if (!p.granted[i]) continue;
            const int now = fork_row(p, i, lane, kWave);
            if (lane == 0) p.held[p.dst[i]] = now;  // read by this wave only
        }
    }
}

// One workgroup per fork.
__global__ __launch_bounds__(kPoolThreads) void fork_apply_kernel(PoolParams p) {
    const int i = blockIdx.x;
    if (!p.granted[i]) return;
    const int now = fork_row(p, i, threadIdx.x, kPoolThreads);
    __syncthreads();  // every thread has read held
    if (threadIdx.x == 0) p.held[p.dst[i]] = now;
}

// Copies `slots` slots of a page in every layer, keys and values: an item is one
// T of one (head, slot), eight of them on their way a thread. Bound by bytes: 224 pages
// of 8 layers, 451 MB read and written, take 91 us, 5.0 TB/s.
template <typename T>
__global__ __launch_bounds__(kCopyThreads) void copy_pages_kernel(PageMoveParams p) {
    const int src = p.src[blockIdx.x], dst = p.dst[blockIdx.x];
    if (src < 0 || src >= p.pages || dst < 0 || dst >= p.pages || src == dst) return;
    const int slots = p.slots ? clamped(p.slots[blockIdx.x], 0, p.page) : p.page;
    const int row = p.row_bytes / (int)sizeof(T);
    const int64_t items = (int64_t)p.heads * slots * row;
    char *base = static_cast<char *>(blockIdx.y & 1 ? p.v : p.k) +
                 (int64_t)(blockIdx.y >> 1) * p.layer_stride;
    const char *in = base + (int64_t)src * p.page_stride;
    char *out = base + (int64_t)dst * p.page_stride;
    constexpr int kAhead = 8;
    const int64_t stride = (int64_t)gridDim.z * kCopyThreads;
    for (int64_t i0 = (int64_t)blockIdx.z * kCopyThreads + threadIdx.x; i0 < items;
         i0 += stride * kAhead) {
        T x[kAhead];
        int64_t at[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t i = i0 + u * stride;
            at[u] = -1;
            if (i < items) {
                const int64_t hs = udiv64(i, row), h = udiv64(hs, slots);
                at[u] = h * p.head_stride + (hs - h * slots) * p.slot_stride +
                        (i - hs * row) * (int64_t)sizeof(T);
                x[u] = *reinterpret_cast<const T *>(in + at[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (at[u] >= 0) *reinterpret_cast<T *>(out + at[u]) = x[u];
    }
}

// Brings an accepted path together: position ctx + i takes what stands at ctx +
// path[i]. A thread owns the same T of every position and layer, and path[i] >= i
// rises, so eight positions may be read before any of them is written, and no
// later one is written over before it is read. 256 requests in 16 layers, 34 MB read and
// written, take 11 us: four dependent reads (count, path, table, keys) and the launch.
template <typename T>
__global__ __launch_bounds__(kMoveThreads) void move_kv_kernel(PageMoveParams p) {
    __shared__ int64_t from_s[kMoveThreads], to_s[kMoveThreads];
    const int b = blockIdx.x;
    int n = p.accepted[b];
    n = n < p.width - 1 ? n : p.width - 1;
    if (n < 1) return;
    const int64_t ctx = p.ctx[b] < 0 ? 0 : p.ctx[b];
    const int32_t *table = p.c.table + (int64_t)b * p.c.table_width;
    char *base = static_cast<char *>(blockIdx.y & 1 ? p.v : p.k) +
                 (int64_t)(blockIdx.y >> 1) * p.layer_stride;
    const int row = p.row_bytes / (int)sizeof(T);
    auto offset = [&](int64_t pos) {
        return pos > 0x7FFFFFFF ? (int64_t)-1 : slot_offset(p.c, table, (int)pos, 0);
    };
    for (int i0 = 1; i0 <= n; i0 += kMoveThreads) {
        __syncthreads();
        const int i = i0 + threadIdx.x;
        int64_t from = -1, to = -1;
        if (i <= n) {
            const int j = p.path[(int64_t)b * p.width + i];
            if (j >= 0 && j != i) {
                from = offset(ctx + j);
                to = offset(ctx + i);
            }
        }
        from_s[threadIdx.x] = to < 0 ? -1 : from;
        to_s[threadIdx.x] = to;
        __syncthreads();
        const int m = n - i0 + 1 < kMoveThreads ? n - i0 + 1 : kMoveThreads;
        for (int x = blockIdx.z * kMoveThreads + threadIdx.x; x < p.heads * row;
             x += gridDim.z * kMoveThreads) {
            const int h = x / row;
            char *at = base + h * p.head_stride + (int64_t)(x - h * row) * (int64_t)sizeof(T);
            constexpr int kAhead = 8;
            for (int k = 0; k < m; k += kAhead) {
                T y[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (k + u < m && from_s[k + u] >= 0)
                        y[u] = *reinterpret_cast<const T *>(at + from_s[k + u]);
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (k + u < m && from_s[k + u] >= 0)
                        *reinterpret_cast<T *>(at + to_s[k + u]) = y[u];
            }
        }
    }
}

hipError_t launch_resize_pages(const PoolParams &p, hipStream_t s) {
    hipLaunchKernelGGL(resize_pages_kernel, dim3(1), dim3(kPoolThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_fork_pages(const PoolParams &p, hipStream_t s) {
    // One launch for as many forks as waves, of short rows: three forks take 6.6 us so,
    // 9.4 in two launches, which longer rows need to be spread over the device.
    if (p.n <= kPoolWaves && p.width <= 4 * kWave) {
        hipLaunchKernelGGL((fork_plan_kernel<true>), dim3(1), dim3(kPoolThreads), 0, s, p);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((fork_plan_kernel<false>), dim3(1), dim3(kPoolThreads), 0, s, p);
    hipLaunchKernelGGL(fork_apply_kernel, dim3((unsigned)p.n), dim3(kPoolThreads), 0, s, p);
    return hipGetLastError();
}

// The widest access that every row of the pools is aligned to.
static int access_bytes(const PageMoveParams &p) {
    const uint64_t all = (uint64_t)(uintptr_t)p.k | (uint64_t)(uintptr_t)p.v |
                         (uint64_t)p.layer_stride | (uint64_t)p.page_stride |
                         (uint64_t)p.head_stride | (uint64_t)p.slot_stride | (uint64_t)p.row_bytes;
    return all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : 1);
}

hipError_t launch_copy_pages(const PageMoveParams &p, hipStream_t s) {
    auto go = [&](auto unit) {
        using T = decltype(unit);
        const int64_t items = (int64_t)p.heads * p.page * (p.row_bytes / (int)sizeof(T));
        int64_t split = (items + 8 * kCopyThreads - 1) / (8 * kCopyThreads);
        split = split < 64 ? split : 64;
        hipLaunchKernelGGL((copy_pages_kernel<T>),
                           dim3((unsigned)p.n, (unsigned)(2 * p.layers), (unsigned)split),
                           dim3(kCopyThreads), 0, s, p);
    };
    switch (access_bytes(p)) {
    case 16: go(u32x4()); break;
    case 4: go(uint32_t()); break;
    default: go(uint8_t());
    }
    return hipGetLastError();
}

hipError_t launch_move_kv(const PageMoveParams &p, hipStream_t s) {
    PageMoveParams q = p;
    auto go = [&](auto unit) {
        using T = decltype(unit);
        const int items = p.heads * (p.row_bytes / (int)sizeof(T));
        int split = (items + kMoveThreads - 1) / kMoveThreads;
        split = split < 64 ? split : 64;
        hipLaunchKernelGGL((move_kv_kernel<T>),
                           dim3((unsigned)p.n, (unsigned)(2 * p.layers), (unsigned)split),
                           dim3(kMoveThreads), 0, s, q);
    };
    switch (access_bytes(p)) {
    case 16: go(u32x4()); break;
    case 4: go(uint32_t()); break;
    default: go(uint8_t());
    }
    return hipGetLastError();
}

}  // namespace dspark
