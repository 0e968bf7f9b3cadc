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
constexpr int kPerThread = 16;  // entries of refs that a thread looks at together
constexpr int kMoveThreads = 128;
constexpr int kCopyThreads = 256;

// What threads of the workgroup have written is read anew afterwards, past the
// vector cache: the atomics on refs do not go through it.
__device__ __forceinline__ void pool_barrier() {
    __threadfence();
    __syncthreads();
    __threadfence();
}

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

// Takes the lowest free pages from `from` (a multiple of the workgroup's share) on:
// take(rank, page) is called for ranks 0 .. need - 1 as far as there are free pages.
// Returns how many there were; `from` is left where the next search goes on.
template <typename Take>
__device__ __forceinline__ int take_free(int32_t *refs, int pages, int &from, int need, int *lds,
                                         Take take) {
    int found = 0;
    while (found < need && from < pages) {
        const int p0 = from + threadIdx.x * kPerThread;
        int32_t r[kPerThread];
        int zeros = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) r[i] = p0 + i < pages ? refs[p0 + i] : 1;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) zeros += r[i] == 0;
        int all;
        int rank = found + pool_scan(zeros, lds, all) - zeros;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            if (r[i] != 0) continue;
            if (rank < need) {
                refs[p0 + i] = 1;
                take(rank, p0 + i);
            }
            ++rank;
        }
        found += all;
        if (found <= need) from += kPoolThreads * kPerThread;
    }
    pool_barrier();
    return found < need ? found : need;
}

// The last index b of a non-decreasing LDS array [n] with before[b] <= x.
__device__ __forceinline__ int owner(const int *before, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One workgroup, 1024 rows at a time: first every row's pages past its length are
// released, then the rows that need more take theirs. Both work on the entries of
// all rows laid end to end, so one long row costs no more than many short ones.
__global__ __launch_bounds__(kPoolThreads) void resize_pages_kernel(PoolParams p) {
    __shared__ int before_s[kPoolThreads], held_s[kPoolThreads], lds[kPoolWaves];
    auto rows_from = [&](int b0, int &held, int &want) {
        const int b = b0 + threadIdx.x;
        held = want = 0;
        if (b >= p.R) return;
        held = clamped(p.held[b], 0, p.width);
        const int64_t len = p.lens[b] < 0 ? 0 : p.lens[b];
        const int64_t n = (len + p.page - 1) / p.page;
        want = n > p.width ? -1 : (int)n;  // more than a row can hold: not served
    };
    for (int b0 = 0; b0 < p.R; b0 += kPoolThreads) {
        int held, want, all;
        rows_from(b0, held, want);
        const int less = want >= 0 && held > want ? held - want : 0;
        const int in = pool_scan(less, lds, all);
        before_s[threadIdx.x] = in - less;
        held_s[threadIdx.x] = want;
        __syncthreads();
        for (int i = threadIdx.x; i < all; i += kPoolThreads) {
            const int b = owner(before_s, kPoolThreads, i);
            int32_t *e = p.table + (int64_t)(b0 + b) * p.width + held_s[b] + (i - before_s[b]);
            release(p.refs, p.pages, *e);
            *e = -1;
        }
        if (less > 0) p.held[b0 + threadIdx.x] = want;
        if (b0 + (int)threadIdx.x < p.R) p.granted[b0 + threadIdx.x] = want >= 0;
        __syncthreads();
    }
    pool_barrier();
    int from = 0;
    bool short_of = false;
    for (int b0 = 0; b0 < p.R; b0 += kPoolThreads) {
        int held, want, all;
        rows_from(b0, held, want);
        const int more = want > held ? want - held : 0;
        const int in = pool_scan(more, lds, all);
        if (all == 0) continue;
        before_s[threadIdx.x] = in - more;
        held_s[threadIdx.x] = held;
        __syncthreads();
        auto entry = [&](int rank) {
            const int b = owner(before_s, kPoolThreads, rank);
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
            const int first = before_s[owner(before_s, kPoolThreads, got)];
            for (int rank = first + threadIdx.x; rank < got; rank += kPoolThreads) {
                int32_t *e = entry(rank);
                release(p.refs, p.pages, *e);
                *e = -1;
            }
            short_of = true;
        }
        pool_barrier();
    }
}

// One workgroup: which forks are granted, and a fresh page for each that ends
// inside a page.
__global__ __launch_bounds__(kPoolThreads) void fork_plan_kernel(PoolParams p) {
    __shared__ int src_s[kPoolThreads], dst_s[kPoolThreads], fresh_s[kPoolThreads], lds[kPoolWaves];
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
            src_s[threadIdx.x] = k < p.n ? p.src[k] : -1;
            dst_s[threadIdx.x] = k < p.n ? p.dst[k] : -1;
            __syncthreads();
            const int m = p.n - k0 < kPoolThreads ? p.n - k0 : kPoolThreads;
            for (int u = 0; u < m; ++u) ok &= d != src_s[u] && (d != dst_s[u] || k0 + u >= i);
        }
        int part = -1, rest = 0;
        if (ok) {
            const int held = clamped(p.held[s], 0, p.width);
            const int64_t most = (int64_t)held * p.page;
            int64_t len = p.lens[s] < 0 ? 0 : p.lens[s];
            len = len < most ? len : most;
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
}

// One workgroup per fork: the target's old pages go, the source's full pages and the
// fresh one come. The source keeps its own hold on what is shared, so no page looks
// free in between, whatever the order.
__global__ __launch_bounds__(kPoolThreads) void fork_apply_kernel(PoolParams p) {
    const int i = blockIdx.x;
    if (!p.granted[i]) return;
    const int s = p.src[i], d = p.dst[i], fresh = p.copy_dst[i];
    if (s < 0 || s >= p.R || d < 0 || d >= p.R) return;
    const int held = clamped(p.held[s], 0, p.width), old = clamped(p.held[d], 0, p.width);
    const int64_t most = (int64_t)held * p.page;
    int64_t len = p.lens[s] < 0 ? 0 : p.lens[s];
    len = len < most ? len : most;
    const int full = (int)(len / p.page), now = full + (fresh >= 0);
    const int32_t *in = p.table + (int64_t)s * p.width;
    int32_t *out = p.table + (int64_t)d * p.width;
    const int last = now > old ? now : old;
    for (int e = threadIdx.x; e < last; e += kPoolThreads) {
        const int page = e < full ? in[e] : (e < now ? fresh : -1);
        if (e < full && page >= 0 && page < p.pages) atomicAdd(p.refs + page, 1);
        if (e < old) release(p.refs, p.pages, out[e]);
        out[e] = page;
    }
    __syncthreads();  // every thread has read held[d]
    if (threadIdx.x == 0) p.held[d] = now;
}

// Copies `slots` slots of a page in every layer, keys and values: an item is one
// T of one (head, slot), eight of them on their way a thread.
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
// later one is written over before it is read.
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
    hipLaunchKernelGGL(fork_plan_kernel, dim3(1), dim3(kPoolThreads), 0, s, p);
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
