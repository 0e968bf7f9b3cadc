// sample.hip - the target's token of every packed verify row, drawn with the
// request's temperature, top-k, top-p and min-p from a given uniform number,
// then acceptance and bonus of every request.
//
// A row's logits are ranked by value, lowest index first among equals, and
// weigh w = exp((x - max) / T). The filters each keep a prefix of that order:
// the first k; the entries whose preceding weight is below p of the kept sum;
// those with w >= min_p. The draw takes the first entry whose cumulated weight
// exceeds u times the kept sum.
//
// bf16 leaves few distinct values, so a row is a histogram: the count of every
// value holds all that the filters and the draw need, exactly, and the weights
// are taken in 64 bits once per value. The border of a cut then moves by 1e-15
// of the sum where a sum of fp32 weights moves it by 1e-6, which at 1e5 entries
// would change the drawn token of several rows in a hundred.
#include "argmax_dev.hpp"
#include "forward.hpp"

namespace dspark {

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / kWave;
constexpr int kBins = 32768;      // counters resident at once: half of the key range
constexpr int kChunks = 1024;     // of 64 neighbouring values each

// Order-preserving 16-bit key of a bf16 value, -0 on +0.
__device__ __forceinline__ uint32_t value_key(uint32_t bits) {
    if (bits == 0x8000u) bits = 0;
    return bits & 0x8000u ? (~bits & 0xFFFFu) : (bits | 0x8000u);
}
__device__ __forceinline__ double key_value(uint32_t key) {
    const uint32_t bits = key & 0x8000u ? key ^ 0x8000u : ~key & 0xFFFFu;
    return (double)bf16_f32((uint16_t)bits);
}
// Keys that take part: NaN and -inf weigh nothing.
__device__ __forceinline__ bool key_counts(uint32_t key) { return key >= 0x80u && key <= 0xFF80u; }

// f(key, index) for every entry of a row, by the whole workgroup.
template <bool kVec, typename F>
__device__ __forceinline__ void for_row(const uint16_t *__restrict__ row, int V, F f) {
    if (kVec) {
        const u32x4 *r4 = reinterpret_cast<const u32x4 *>(row);
        for (int v = threadIdx.x; v < V / 8; v += kSampleThreads) {
            const u32x4 a = r4[v];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f(value_key(a[i] & 0xFFFFu), 8 * v + 2 * i);
                f(value_key(a[i] >> 16), 8 * v + 2 * i + 1);
            }
        }
    } else {
        for (int v = threadIdx.x; v < V; v += kSampleThreads) f(value_key(row[v]), v);
    }
}

__device__ __forceinline__ double wave_incl_sum(double x) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const double y = __shfl_up(x, off, kWave);
        if (lane >= off) x += y;
    }
    return x;
}

struct SampleLds {
    uint32_t bins[kBins];
    double wex[kChunks];   // weight and count before each chunk, descending order
    int cex[kChunks];
    double wpart[kSampleWaves];
    int cpart[kSampleWaves];
    uint32_t detail[kWave];  // counts of one chunk
    uint32_t top;            // largest key that counts, 0 if none
    int at, count;
    double total;
};

template <bool kVec>
__global__ __launch_bounds__(kSampleThreads) void sample_rows_kernel(SampleParams p) {
    __shared__ SampleLds s;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int cap = p.B * (p.gamma + 1);
    const int r = blockIdx.x;
    if (r >= packed_total(p.cu, p.B, cap)) return;
    const int b = wave_request_of(p.cu, p.B, r);
    if (b >= p.B || r < p.cu[0]) return;
    const int src = p.psrc ? p.psrc[r] : r;
    if (src < 0 || src >= cap) {
        if (tid == 0) p.sample[r] = -1;
        return;
    }
    const uint16_t *row = p.logits + (int64_t)src * p.V;
    const double T = p.temperature ? (double)p.temperature[b] : 1.0;
    const int k = p.top_k ? p.top_k[b] : 0;
    const double top_p = p.top_p ? (double)p.top_p[b] : 1.0;
    const double min_p = p.min_p ? (double)p.min_p[b] : 0.0;
    const double u = p.uniforms[r] > 0.f ? (double)p.uniforms[r] : 0.0;

    if (tid == 0) s.top = 0;
    __syncthreads();
    uint32_t best = 0;
    for_row<kVec>(row, p.V, [&](uint32_t key, int) {
        if (key_counts(key)) best = key > best ? key : best;
    });
    atomicMax(&s.top, best);
    __syncthreads();
    const uint32_t top = s.top;

    // the (j+1)-th entry, in index order, that holds `key`: each wave counts its
    // own contiguous share, then the share that holds it is searched
    auto index_of = [&](uint32_t key, int j) -> int {
        const int per = (p.V + kSampleWaves - 1) / kSampleWaves;
        const int lo = wave * per, hi = lo + per < p.V ? lo + per : p.V;
        int n = 0;
        for (int v = lo + lane; v < hi; v += kWave) n += value_key(row[v]) == key;
#pragma unroll
        for (int off = kWave / 2; off > 0; off >>= 1) n += __shfl_xor(n, off, kWave);
        if (lane == 0) s.cpart[wave] = n;
        if (tid == 0) s.at = 0;
        __syncthreads();
        int before = 0;
        for (int i = 0; i < wave; ++i) before += s.cpart[i];
        if (j >= before && j < before + n) {
            for (int v0 = lo; v0 < hi; v0 += kWave) {
                const bool hit = v0 + lane < hi && value_key(row[v0 + lane]) == key;
                const uint64_t m = __ballot(hit);
                const int mine = before + __popcll(m & ((1ull << lane) - 1));
                if (hit && mine == j) s.at = v0 + lane;
                before += __popcll(m);
                if (before > j) break;
            }
        }
        __syncthreads();
        return s.at;
    };
    if (top == 0 || !(T > 0.0)) {  // greedy, or nothing to draw from: the lowest index
        const int at = top == 0 ? 0 : index_of(top, 0);
        if (tid == 0) p.sample[r] = at;
        return;
    }
    const double vmax = key_value(top);
    auto weight = [&](uint32_t key) { return key == top ? 1.0 : exp((key_value(key) - vmax) / T); };

    // count and weight of every chunk: thread t owns chunk 1023 - t
    int cnt = 0;
    double wsum = 0.0;
    for (int half = 1; half >= 0; --half) {
        for (int i = tid; i < kBins; i += kSampleThreads) s.bins[i] = 0;
        __syncthreads();
        for_row<kVec>(row, p.V, [&](uint32_t key, int) {
            if (key_counts(key) && (int)(key >> 15) == half) atomicAdd(&s.bins[key & (kBins - 1)], 1u);
        });
        __syncthreads();
        const int chunk = kChunks - 1 - tid;
        if (chunk >> 9 == half) {
            for (int i = 63; i >= 0; --i) {
                const uint32_t key = (uint32_t)chunk * 64 + i;
                const uint32_t n = s.bins[key & (kBins - 1)];
                if (n) {
                    cnt += (int)n;
                    wsum += (double)n * weight(key);
                }
            }
        }
        __syncthreads();
    }
    // exclusive prefixes over the chunks
    int ci = wave_incl_scan(cnt, lane);
    double wi = wave_incl_sum(wsum);
    if (lane == kWave - 1) {
        s.cpart[wave] = ci;
        s.wpart[wave] = wi;
    }
    __syncthreads();
    for (int i = 0; i < wave; ++i) {
        ci += s.cpart[i];
        wi += s.wpart[i];
    }
    s.cex[tid] = ci - cnt;
    s.wex[tid] = wi - wsum;
    if (tid == kSampleThreads - 1) {
        s.count = ci;
        s.total = wi;
    }
    __syncthreads();
    // the prefix sum as the next chunk sees it, the same number for both
    const int c0 = s.cex[tid], c1 = tid + 1 < kChunks ? s.cex[tid + 1] : s.count;
    const double w0 = s.wex[tid], w1 = tid + 1 < kChunks ? s.wex[tid + 1] : s.total;
    int N = s.count;
    double total = s.total;

    // The chunk at descending place t: lane l of every wave gets the count n and
    // weight w of its (l+1)-th largest value and what precedes it.
    int have = -1;
    int n = 0, cb = 0;
    double w = 0.0, eb = 0.0;
    auto detail = [&](int t) {
        if (t != have) {
            __syncthreads();
            if (tid < kWave) s.detail[tid] = 0;
            __syncthreads();
            const uint32_t chunk = (uint32_t)(kChunks - 1 - t);
            for_row<kVec>(row, p.V, [&](uint32_t key, int) {
                if (key_counts(key) && key >> 6 == chunk) atomicAdd(&s.detail[key & 63], 1u);
            });
            __syncthreads();
            n = (int)s.detail[63 - lane];
            w = n ? weight(chunk * 64 + 63 - lane) : 0.0;
            cb = s.cex[t] + wave_incl_scan(n, lane) - n;
            const double x = (double)n * w;
            eb = s.wex[t] + (wave_incl_sum(x) - x);
            have = t;
        }
    };
    // the place of the one thread for which `here` holds (-1 if none)
    auto place = [&](bool here) {
        __syncthreads();
        if (tid == 0) s.at = -1;
        __syncthreads();
        if (here) s.at = tid;
        __syncthreads();
        return s.at;
    };
    auto wave_sum_int = [&](int x) {
#pragma unroll
        for (int off = kWave / 2; off > 0; off >>= 1) x += __shfl_xor(x, off, kWave);
        return x;
    };
    // keeps the first `keep` entries, which end inside the chunk at hand
    auto cut = [&](int keep) {
        keep = keep < 1 ? 1 : keep;
        if (keep >= N) return;
        const int t = place(c0 < keep && keep <= c1);
        detail(t);
        int mine = keep - cb;
        mine = mine < 0 ? 0 : (mine > n ? n : mine);
        const double x = wave_incl_sum((double)mine * w);
        total = s.wex[t] + __shfl(x, kWave - 1, kWave);
        N = keep;
    };
    if (k > 0) cut(k);
    if (top_p < 1.0) {
        const double goal = top_p * total;
        const int t = place(c1 > c0 && w0 < goal && !(w1 < goal));
        if (t >= 0) {
            detail(t);
            int m = 0;
            if (n && eb < goal) {
                m = n;
                if (w > 0.0) {
                    const double q = ceil((goal - eb) / w);
                    m = q < (double)n ? (int)q : n;
                    while (m > 0 && !(eb + (double)(m - 1) * w < goal)) --m;
                    while (m < n && eb + (double)m * w < goal) ++m;
                }
            }
            cut(s.cex[t] + wave_sum_int(m));
        } else if (!(goal > 0.0)) {
            cut(1);
        }
    }
    if (min_p > 0.0) {
        const uint32_t low = (uint32_t)(kChunks - 1 - tid) * 64;
        const bool whole = c1 > c0 && weight(low < 0x80u ? 0x80u : low) >= min_p;
        // the first chunk that is not kept whole: no earlier one with entries fails
        const int t = place(false);
        (void)t;
        if (c1 > c0 && !whole) atomicMin((unsigned *)&s.at, (unsigned)tid);  // -1 is the largest
        __syncthreads();
        const int f = s.at;
        if (f >= 0) {
            detail(f);
            cut(s.cex[f] + wave_sum_int(n && w >= min_p ? n : 0));
        }
    }
    // the draw
    const double goal = u * total;
    int rank = N - 1;
    const int t = place(c1 > c0 && !(w1 <= goal) && w0 <= goal);
    if (t >= 0) {
        detail(t);
        int m = 0;
        if (n && w > 0.0) {
            const double q = floor((goal - eb) / w);
            m = q < 0.0 ? 0 : (q < (double)n ? (int)q : n);
            while (m > 0 && !(eb + (double)m * w <= goal)) --m;
            while (m < n && eb + (double)(m + 1) * w <= goal) ++m;
        }
        const int x = s.cex[t] + wave_sum_int(m);
        rank = x < rank ? x : rank;
    }
    const int at = place(c0 <= rank && rank < c1);
    detail(at);
    __syncthreads();
    if (wave == 0 && cb <= rank && rank < cb + n) {
        s.count = rank - cb;
        s.top = (uint32_t)(kChunks - 1 - at) * 64 + 63 - lane;
    }
    __syncthreads();
    const int chosen = index_of(s.top, s.count);
    if (tid == 0) p.sample[r] = chosen;
}

__global__ __launch_bounds__(256) void sample_finish_kernel(SampleParams p) {
    const int b = blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave;
    if (b >= p.B) return;
    const int cap = p.B * (p.gamma + 1);
    const int total = packed_total(p.cu, p.B, cap);
    int start = p.cu[b], end = p.cu[b + 1];
    start = start < 0 ? 0 : (start > total ? total : start);
    end = end < start ? start : (end > total ? total : end);
    wave_accept_rows([&](int j) { return p.sample[start + j]; }, end - start, p.gamma,
                     p.tokens + (int64_t)b * (p.gamma + 1), p.sample + start, p.acc + b,
                     p.bonus + b);
}

hipError_t launch_sample_accept(const SampleParams &p, void *ws, hipStream_t s) {
    (void)ws;
    const int cap = p.B * (p.gamma + 1);
    const bool vec = p.V % 8 == 0 && (uintptr_t)p.logits % 16 == 0;
    if (vec) hipLaunchKernelGGL((sample_rows_kernel<true>), dim3(cap), dim3(kSampleThreads), 0, s, p);
    else hipLaunchKernelGGL((sample_rows_kernel<false>), dim3(cap), dim3(kSampleThreads), 0, s, p);
    const int wpb = 256 / kWave;
    hipLaunchKernelGGL(sample_finish_kernel, dim3((p.B + wpb - 1) / wpb), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace dspark
