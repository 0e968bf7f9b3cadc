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

constexpr int kSampleThreads = 512;
constexpr int kSampleWaves = kSampleThreads / kWave;
constexpr int kSampleWavesPerSimd = 6;  // three workgroups a CU
constexpr int kRowUnroll = 8;  // 16-byte loads in flight per lane

// Places. A value's place counts down the ranking; 64 places are a block.
//
// Narrow places: |x| in [2^-32, 2^16), 128 values an octave and a sign, one
// place each, with a place for what is larger or smaller at every end. The
// counters of all of them take 48 KiB of LDS, so three workgroups share a CU
// and one's loads run beside another's atomics. The end places hold more than
// one value, so a row is finished this way only if they do not matter: nothing
// at or above 2^16, nothing nonzero below 2^-32, and what lies at or below
// -2^16 (masks, -inf) so far down that it weighs nothing (kNegligible).
//
// Wide places: every bf16 value, 65536 places, counted in eight rounds over
// the row. Any row can be finished this way.
constexpr uint32_t kNarrowLo = (127 - 32) << 7, kNarrowHi = (127 + 16) << 7;  // bits of |x|
constexpr int kNarrowSpan = (int)(kNarrowHi - kNarrowLo);
constexpr int kPlaceZero = kNarrowSpan + 1;  // +0 and what is below 2^-32
constexpr int kPlaceMinus = kPlaceZero + 1;  // -0 and what is above -2^-32
constexpr int kPlaceLow = kPlaceMinus + kNarrowSpan + 1;  // -2^16 and below, NaN
constexpr int kNarrowBlocks = (kPlaceLow + kWave) / kWave;
constexpr int kWideBlocks = 1024;
constexpr int kWideRound = 8192;  // counters of one round
// exp(-60) of the largest weight times 2^31 entries is 2e-17 of the sum, below
// the half step of the 64-bit sums.
constexpr double kNegligible = 60.0;

struct Narrow {
    static constexpr int kBlocks = kNarrowBlocks;
    uint32_t bins[kBlocks * kWave];
    double wex[kBlocks + 1];  // weight and count before each block
    int cex[kBlocks + 1];
    // bits of the value at a place
    __device__ static uint32_t bits(int e) {
        e = e > kPlaceLow ? kPlaceLow : e;
        if (e == kPlaceZero || e == kPlaceMinus) return 0u;
        return e < kPlaceZero ? kNarrowHi - (uint32_t)e
                              : 0x8000u | (kNarrowLo - 1u + (uint32_t)(e - kPlaceMinus));
    }
};
struct Wide {
    static constexpr int kBlocks = kWideBlocks;
    uint32_t bins[kWideRound];
    uint32_t detail[kWave];  // counts of the block at hand
    double wex[kBlocks + 1];
    int cex[kBlocks + 1];
    __device__ static uint32_t bits(int e) {
        const uint32_t key = 0xFFFFu - (uint32_t)e;
        return key & 0x8000u ? key ^ 0x8000u : ~key & 0xFFFFu;
    }
};
struct SampleLds {
    union {
        Narrow narrow;
        Wide wide;
    };
    int part[kSampleWaves];
    unsigned top;  // place of the largest value that counts
    int flag, at;
};

// Order-preserving 16-bit key of a bf16 value, -0 on +0; the keys that take
// part: NaN and -inf weigh nothing.
__device__ __forceinline__ uint32_t value_key(uint32_t bits) {
    if (bits == 0x8000u) bits = 0;
    return bits & 0x8000u ? (~bits & 0xFFFFu) : (bits | 0x8000u);
}
__device__ __forceinline__ bool key_counts(uint32_t key) { return key >= 0x80u && key <= 0xFF80u; }

// A row as 16-byte vectors, with up to 7 entries before and after them.
struct Row {
    const uint16_t *p;
    int V, head, vecs;
    __device__ Row(const uint16_t *at, int n) : p(at), V(n) {
        head = (int)((16 - ((uintptr_t)at & 15)) & 15) / 2;
        head = head < n ? head : n;
        vecs = (n - head) / 8;
    }
    __device__ int loose() const { return V - 8 * vecs; }
    // index of the i-th entry outside the vectors
    __device__ int loose_at(int i) const { return i < head ? i : 8 * vecs + i; }
    __device__ const u32x4 *vec() const { return reinterpret_cast<const u32x4 *>(p + head); }
};

// f(vector, its number) for vectors [v0, v1), by lanes `step` apart, the first
// of them at v0 + lane; f must take lanes that are off.
template <typename F>
__device__ __forceinline__ void for_vecs(const Row &row, int v0, int v1, int lane, int step, F f) {
    const u32x4 *at = row.vec();
    int v = v0 + lane;
    for (; v + (kRowUnroll - 1) * step < v1; v += kRowUnroll * step) {
        u32x4 a[kRowUnroll];
#pragma unroll
        for (int i = 0; i < kRowUnroll; ++i) a[i] = at[v + i * step];
#pragma unroll
        for (int i = 0; i < kRowUnroll; ++i) f(a[i], v + i * step);
    }
    if (v < v1) {  // the last round's loads past the end repeat its first
        u32x4 a[kRowUnroll];
#pragma unroll
        for (int i = 0; i < kRowUnroll; ++i) a[i] = at[v + i * step < v1 ? v + i * step : v];
#pragma unroll
        for (int i = 0; i < kRowUnroll; ++i)
            if (v + i * step < v1) f(a[i], v + i * step);
    }
}
// f(bits) for every entry of the row, by the whole workgroup.
template <typename F>
__device__ __forceinline__ void for_row(const Row &row, F f) {
    for_vecs(row, 0, row.vecs, threadIdx.x, kSampleThreads, [&](u32x4 a, int) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f(a[i] & 0xFFFFu);
            f(a[i] >> 16);
        }
    });
    if ((int)threadIdx.x < row.loose()) f((uint32_t)row.p[row.loose_at(threadIdx.x)]);
}

// Byte offsets of the counters of two values' narrow places, packed.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t narrow_offsets(uint32_t two) {
    constexpr unsigned short lo = kNarrowLo - 1, hi = kNarrowHi;
    const u16x2 x = __builtin_bit_cast(u16x2, two);
    u16x2 m = __builtin_bit_cast(u16x2, two & 0x7FFF7FFFu);
    m = __builtin_elementwise_max(m, (u16x2){lo, lo});
    m = __builtin_elementwise_min(m, (u16x2){hi, hi}) - (u16x2){lo, lo};
    // the place is kPlaceZero - m for a positive value, kPlaceMinus + m for a negative one
    const u16x2 sign = __builtin_bit_cast(u16x2, __builtin_bit_cast(i16x2, x) >> 15);
    const u16x2 e = (u16x2){kPlaceMinus, kPlaceMinus} + (m ^ ~sign);
    return __builtin_bit_cast(uint32_t, (u16x2)(e << 2));
}

// Inclusive sum over the wave, lane 0 first, by the DPP moves of wave_incl_scan.
__device__ __forceinline__ double wave_incl_sum(double x) {
    auto moved = [](double v, auto move) {
        const uint64_t u = (uint64_t)__double_as_longlong(v);
        const uint32_t lo = move((uint32_t)u), hi = move((uint32_t)(u >> 32));
        return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
    };
    x += moved(x, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x111, 0xF, 0xF, false); });
    x += moved(x, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x112, 0xF, 0xF, false); });
    x += moved(x, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x114, 0xF, 0xF, false); });
    x += moved(x, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x118, 0xF, 0xF, false); });
    x += moved(x, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x142, 0xA, 0xF, false); });
    x += moved(x, [](uint32_t w) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x143, 0xC, 0xF, false); });
    return x;
}
__device__ __forceinline__ double last_lane(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, kWave - 1);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), kWave - 1);
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ int last_lane(int x) { return __builtin_amdgcn_readlane(x, kWave - 1); }

struct Draw {
    double T, u, top_p, min_p;
    int k;
};
// What a row draws: the bits of its value, and which of its n equals.
struct Drawn {
    uint32_t bits;
    int j, n;
};

// Counts and weights of all blocks are in place (prefix sums in wex and cex,
// totals at their ends); every wave walks the filters by itself, with the
// same numbers. counts(t) gives lane l the count of place 64*t + l.
template <typename H, typename Weight, typename Counts>
__device__ __forceinline__ Drawn walk_filters(const H &h, const Draw &d, Weight weight,
                                              Counts counts) {
    const int lane = threadIdx.x & (kWave - 1);
    // the first block for which `test` holds, -1 if none
    auto first = [&](auto test) {
        for (int i0 = 0; i0 < H::kBlocks; i0 += kWave) {
            const int i = i0 + lane;
            const uint64_t m = __ballot(i < H::kBlocks && test(i));
            if (m) return i0 + __ffsll((unsigned long long)m) - 1;
        }
        return -1;
    };
    // count and weight of this lane's place in block t, and what precedes it
    int n = 0, before = 0, have = -1;
    double w = 0.0, ahead = 0.0;
    auto open = [&](int t) {
        if (t == have) return;
        have = t;
        n = counts(t);
        w = n ? weight(t * kWave + lane) : 0.0;
        before = h.cex[t] + wave_incl_scan(n, lane) - n;
        const double x = (double)n * w;
        ahead = h.wex[t] + (wave_incl_sum(x) - x);
    };
    auto wave_sum = [&](int x) { return last_lane(wave_incl_scan(x, lane)); };
    int N = h.cex[H::kBlocks];
    double total = h.wex[H::kBlocks];
    auto cut = [&](int keep) {
        keep = keep < 1 ? 1 : keep;
        if (keep >= N) return;
        const int t = first([&](int i) { return h.cex[i + 1] >= keep; });
        open(t);
        int mine = keep - before;
        mine = mine < 0 ? 0 : (mine > n ? n : mine);
        total = h.wex[t] + last_lane(wave_incl_sum((double)mine * w));
        N = keep;
    };
    if (d.k > 0) cut(d.k);
    if (d.top_p < 1.0) {
        const double goal = d.top_p * total;
        const int t = goal > 0.0 ? first([&](int i) {
            return h.cex[i + 1] > h.cex[i] && !(h.wex[i + 1] < goal);
        }) : -1;
        if (t >= 0) {
            open(t);
            int m = 0;
            if (n && ahead < goal) {
                m = n;
                if (w > 0.0) {
                    const double q = ceil((goal - ahead) / w);
                    m = q < (double)n ? (int)q : n;
                    while (m > 0 && !(ahead + (double)(m - 1) * w < goal)) --m;
                    while (m < n && ahead + (double)m * w < goal) ++m;
                }
            }
            cut(h.cex[t] + wave_sum(m));
        } else if (!(goal > 0.0)) {
            cut(1);
        }
    }
    if (d.min_p > 0.0) {
        // the first block that is not kept whole
        const int t = first([&](int i) {
            return h.cex[i + 1] > h.cex[i] && !(weight(i * kWave + kWave - 1) >= d.min_p);
        });
        if (t >= 0) {
            open(t);
            cut(h.cex[t] + wave_sum(n && w >= d.min_p ? n : 0));
        }
    }
    const double goal = d.u * total;
    int rank = N - 1;
    const int t = first([&](int i) {
        return h.cex[i + 1] > h.cex[i] && !(h.wex[i + 1] <= goal);
    });
    if (t >= 0) {
        open(t);
        int m = 0;
        if (n && w > 0.0) {
            const double q = floor((goal - ahead) / w);
            m = q < 0.0 ? 0 : (q < (double)n ? (int)q : n);
            while (m > 0 && !(ahead + (double)m * w <= goal)) --m;
            while (m < n && ahead + (double)(m + 1) * w <= goal) ++m;
        }
        const int x = h.cex[t] + wave_sum(m);
        rank = x < rank ? x : rank;
    }
    const int at = first([&](int i) { return h.cex[i + 1] > rank; });
    open(at);
    const uint64_t mine = __ballot(before <= rank && rank < before + n);
    const int l = __ffsll((unsigned long long)mine) - 1;
    Drawn r;
    r.bits = H::bits(at * kWave + l);
    r.n = __builtin_amdgcn_readlane(n, l);
    r.j = rank - __builtin_amdgcn_readlane(before, l);
    return r;
}

// Count and weight of block i from this lane's counter.
template <typename H, typename Weight>
__device__ __forceinline__ void sum_block(H &h, int i, uint32_t n, Weight weight) {
    const int lane = threadIdx.x & (kWave - 1);
    int c = 0;
    double w = 0.0;
    if (__ballot(n != 0)) {
        c = last_lane(wave_incl_scan((int)n, lane));
        w = last_lane(wave_incl_sum(n ? (double)n * weight(i * kWave + lane) : 0.0));
    }
    if (lane == 0) {
        h.cex[i] = c;
        h.wex[i] = w;
    }
}
// Sums of the blocks to sums before them, by one wave.
template <typename H>
__device__ __forceinline__ void scan_blocks(H &h) {
    const int lane = threadIdx.x & (kWave - 1);
    int c0 = 0;
    double w0 = 0.0;
    for (int i0 = 0; i0 < H::kBlocks; i0 += kWave) {
        const int i = i0 + lane;
        const int c = i < H::kBlocks ? h.cex[i] : 0;
        const double w = i < H::kBlocks ? h.wex[i] : 0.0;
        const int ci = wave_incl_scan(c, lane) + c0;
        const double wi = wave_incl_sum(w) + w0;
        // one number is the end of a block and the start of the next
        const double up = __shfl_up(wi, 1, kWave);
        if (i < H::kBlocks) {
            h.cex[i] = ci - c;
            h.wex[i] = lane ? up : w0;
        }
        c0 = last_lane(ci);
        w0 = last_lane(wi);
    }
    if (lane == 0) {
        h.cex[H::kBlocks] = c0;
        h.wex[H::kBlocks] = w0;
    }
}

// The index of the (j+1)-th of the row's n entries that equal `bits` (zeros of
// either sign are equal).
__device__ __forceinline__ int index_of(SampleLds &s, const Row &row, const Drawn &d) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const uint32_t mask = d.bits == 0 ? 0x7FFF7FFFu : 0xFFFFFFFFu;
    const uint32_t want = d.bits | (d.bits << 16);
    auto equal = [&](uint32_t x) { return (x & mask & 0xFFFFu) == d.bits; };
    // a bit per entry; the usual vector holds none and costs 4 steps per word
    auto matches = [&](u32x4 a) {
        uint32_t t[4], some = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = (a[i] & mask) ^ want;
            some |= (t[i] - 0x00010001u) & ~t[i] & 0x80008000u;
        }
        uint32_t m = 0;
        if (some) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m |= ((t[i] & 0xFFFFu) == 0 ? 1u << (2 * i) : 0u) |
                     (t[i] >> 16 == 0 ? 2u << (2 * i) : 0u);
        }
        return m;
    };
    const bool edge = tid < row.loose() && equal(row.p[row.loose_at(tid)]);
    if (d.n == 1) {
        if (edge) s.at = row.loose_at(tid);
        for_vecs(row, 0, row.vecs, tid, kSampleThreads, [&](u32x4 a, int v) {
            const uint32_t m = matches(a);
            if (m) s.at = row.head + 8 * v + __ffs((int)m) - 1;
        });
        __syncthreads();
        return s.at;
    }
    // a contiguous share of the vectors per wave
    const int per = (row.vecs + kSampleWaves - 1) / kSampleWaves;
    const int v0 = wave * per < row.vecs ? wave * per : row.vecs;
    const int v1 = v0 + per < row.vecs ? v0 + per : row.vecs;
    int c = 0;
    for_vecs(row, v0, v1, lane, kWave, [&](u32x4 a, int) { c += __popc(matches(a)); });
    c = last_lane(wave_incl_scan(c, lane));
    if (lane == 0) s.part[wave] = c;
    // the loose entries are all in the first wave: those of the head come first,
    // those of the tail last
    const uint64_t edges = __ballot(edge), heads = edges & ((1ull << row.head) - 1);
    const int place = __popcll((lane < row.head ? heads : edges & ~heads) & ((1ull << lane) - 1));
    if (tid == 0) s.flag = __popcll(heads);
    if (edge && lane < row.head && place == d.j) s.at = lane;
    __syncthreads();
    if (wave == 0) {
        int vectors = 0;
        for (int i = 0; i < kSampleWaves; ++i) vectors += s.part[i];
        if (edge && lane >= row.head && s.flag + vectors + place == d.j)
            s.at = row.loose_at(lane);
    }
    int before = s.flag;
    for (int i = 0; i < wave; ++i) before += s.part[i];
    if (d.j >= before && d.j < before + c) {  // one wave's share at most
        for (int v = v0; v < v1; v += kWave) {
            const uint32_t m = v + lane < v1 ? matches(row.vec()[v + lane]) : 0u;
            const int n = __popc(m), to = before + wave_incl_scan(n, lane);
            if (d.j >= to - n && d.j < to) {
                uint32_t rest = m;
                for (int i = to - n; i < d.j; ++i) rest &= rest - 1;
                s.at = row.head + 8 * (v + lane) + __ffs((int)rest) - 1;
            }
            before = last_lane(to);
            if (before > d.j) break;
        }
    }
    __syncthreads();
    return s.at;
}

// A row with values that the narrow places do not tell apart.
__device__ __forceinline__ Drawn draw_wide(SampleLds &s, const Row &row, const Draw &d) {
    Wide &h = s.wide;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    if (tid == 0) s.top = 0;  // the largest key, here
    __syncthreads();
    uint32_t best = 0;
    for_row(row, [&](uint32_t x) {
        const uint32_t key = value_key(x);
        if (key_counts(key)) best = key > best ? key : best;
    });
    if (best) atomicMax(&s.top, best);
    __syncthreads();
    const uint32_t top = s.top;
    if (top == 0) return Drawn{0u, -1, 0};  // nothing to draw from
    const int first = 0xFFFF - (int)top;
    if (!(d.T > 0.0) || d.k == 1) return Drawn{Wide::bits(first), 0, 2};
    const double vmax = (double)bf16_f32((uint16_t)Wide::bits(first));
    auto weight = [&](int e) {
        return e == first ? 1.0 : exp(((double)bf16_f32((uint16_t)Wide::bits(e)) - vmax) / d.T);
    };
    for (int round = 0; round < 65536 / kWideRound; ++round) {
        for (int i = tid; i < kWideRound; i += kSampleThreads) h.bins[i] = 0;
        __syncthreads();
        for_row(row, [&](uint32_t x) {
            const uint32_t key = value_key(x), e = 0xFFFFu - key;
            if (key_counts(key) && (int)(e / kWideRound) == round)
                atomicAdd(&h.bins[e % kWideRound], 1u);
        });
        __syncthreads();
        for (int i = wave; i < kWideRound / kWave; i += kSampleWaves)
            sum_block(h, round * (kWideRound / kWave) + i, h.bins[i * kWave + lane], weight);
        __syncthreads();
    }
    if (wave == 0) scan_blocks(h);
    __syncthreads();
    return walk_filters(h, d, weight, [&](int t) {
        __syncthreads();
        if (tid < kWave) h.detail[tid] = 0;
        __syncthreads();
        for_row(row, [&](uint32_t x) {
            const uint32_t key = value_key(x), e = 0xFFFFu - key;
            if (key_counts(key) && (int)(e / kWave) == t) atomicAdd(&h.detail[e % kWave], 1u);
        });
        __syncthreads();
        return (int)h.detail[lane];
    });
}

// One workgroup per packed row.
__global__ __launch_bounds__(kSampleThreads, kSampleWavesPerSimd) void sample_rows_kernel(SampleParams p,
                                                                     uint64_t *arrivals) {
    __shared__ SampleLds s;
    Narrow &h = s.narrow;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int cap = p.B * (p.gamma + 1);
    const int r = blockIdx.x;
    const int src = p.psrc ? p.psrc[r] : r;
    const int total = packed_total(p.cu, p.B, cap);
    if (arrivals && r < p.B && p.cu[r + 1] <= p.cu[r] && tid == 0) {  // a request without rows
        p.acc[r] = 0;
        p.bonus[r] = -1;
    }
    if (r >= total) return;
    const bool exists = src >= 0 && src < cap;
    const Row row(p.logits + (int64_t)(exists ? src : 0) * p.V, exists ? p.V : 0);
    for (int i = tid; i < kNarrowBlocks * kWave; i += kSampleThreads) h.bins[i] = 0;
    if (tid == 0) {
        s.top = kNarrowBlocks * kWave;
        s.flag = 0;
    }
    __syncthreads();
    {
        char *bins = reinterpret_cast<char *>(h.bins);
        auto count = [&](uint32_t off) { atomicAdd(reinterpret_cast<uint32_t *>(bins + off), 1u); };
        for_vecs(row, 0, row.vecs, tid, kSampleThreads, [&](u32x4 a, int) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t two = narrow_offsets(a[i]);
                count(two & 0xFFFFu);
                count(two >> 16);
            }
        });
        if (tid < row.loose()) count(narrow_offsets(row.p[row.loose_at(tid)]) & 0xFFFFu);
    }
    const int b = wave_request_of(p.cu, p.B, r);
    Draw d;
    const bool owned = b < p.B && r >= p.cu[0];
    d.T = owned && p.temperature ? (double)p.temperature[b] : 1.0;
    d.k = owned && p.top_k ? p.top_k[b] : 0;
    d.top_p = owned && p.top_p ? (double)p.top_p[b] : 1.0;
    d.min_p = owned && p.min_p ? (double)p.min_p[b] : 0.0;
    d.u = p.uniforms[r] > 0.f ? (double)p.uniforms[r] : 0.0;
    __syncthreads();

    const uint32_t high = h.bins[0], low = h.bins[kPlaceLow];
    const uint32_t zeros = h.bins[kPlaceZero] + h.bins[kPlaceMinus];
    if (zeros) {  // is it only zeros?
        bool small = false;
        for_row(row, [&](uint32_t x) {
            const uint32_t m = x & 0x7FFFu;
            small |= m > 0 && m < kNarrowLo;
        });
        if (small) s.flag = 1;
    }
    __syncthreads();
    if (tid == 0) {
        h.bins[kPlaceZero] = zeros;
        h.bins[kPlaceMinus] = 0;
        h.bins[kPlaceLow] = 0;
    }
    __syncthreads();
    for (int i = wave; i < kNarrowBlocks; i += kSampleWaves) {
        const uint64_t m = __ballot(h.bins[i * kWave + lane] != 0);
        if (m) {
            if (lane == 0) atomicMin(&s.top, (unsigned)(i * kWave + __ffsll((unsigned long long)m) - 1));
            break;
        }
    }
    __syncthreads();
    const int top = (int)s.top;
    const bool small = s.flag != 0;
    const bool greedy = !(d.T > 0.0) || d.k == 1;
    const double vmax = (double)bf16_f32((uint16_t)Narrow::bits(top));
    const bool narrow = high == 0 && !small && top < kPlaceLow &&
                        (low == 0 || greedy || (vmax + 65536.0) / d.T > kNegligible);
    Drawn out;
    if (!exists) {
        out = Drawn{0u, -2, 0};
    } else if (!narrow) {
        __syncthreads();
        out = draw_wide(s, row, d);
    } else if (greedy) {
        out = Drawn{Narrow::bits(top), 0, (int)h.bins[top]};
    } else {
        auto weight = [&](int e) {
            return e == top ? 1.0 : exp(((double)bf16_f32((uint16_t)Narrow::bits(e)) - vmax) / d.T);
        };
        for (int i = wave; i < kNarrowBlocks; i += kSampleWaves)
            sum_block(h, i, h.bins[i * kWave + lane], weight);
        __syncthreads();
        if (wave == 0) scan_blocks(h);
        __syncthreads();
        out = walk_filters(h, d, weight, [&](int t) { return (int)h.bins[t * kWave + lane]; });
    }
    __syncthreads();
    // nothing to draw from: the lowest index; no such source row: -1
    const int chosen = out.j < 0 ? out.j + 1 : index_of(s, row, out);
    if (!owned) return;
    if (!arrivals) {
        if (tid == 0) p.sample[r] = chosen;
        return;
    }
    // the last row of a request to arrive accepts its drafts
    if (wave != 0) return;
    int start = p.cu[b], end = p.cu[b + 1];
    start = start < 0 ? 0 : (start > total ? total : start);
    end = end < start ? start : (end > total ? total : end);
    const int n = end - start;
    bool last = false;
    if (lane == 0) {
        __hip_atomic_store(p.sample + r, chosen, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);  // the token is at the coherence point
        last = __hip_atomic_fetch_add(arrivals + b, (uint64_t)1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) + 1 == (uint64_t)n;
        if (last)  // zero again for the next call
            __hip_atomic_store(arrivals + b, (uint64_t)0, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!__any(last)) return;
    wave_accept_rows(
        [&](int j) {
            return __hip_atomic_load(p.sample + start + j, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
        },
        n, p.gamma, p.tokens + (int64_t)b * (p.gamma + 1), p.sample + start, p.acc + b,
        p.bonus + b);
}

// Acceptance and bonus where the batch has no arrival counters of its own.
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

// One launch up to kMaxFusedB requests (what the workspace counts arrivals
// for), two above.
hipError_t launch_sample_accept(const SampleParams &p, void *ws, hipStream_t s) {
    const int cap = p.B * (p.gamma + 1);
    uint64_t *arrivals = p.B <= kMaxFusedB ? reinterpret_cast<uint64_t *>(static_cast<char *>(ws) +
                                                                          ws_acnt_offset())
                                           : nullptr;
    hipLaunchKernelGGL(sample_rows_kernel, dim3(cap), dim3(kSampleThreads), 0, s, p, arrivals);
    if (!arrivals) {
        const int wpb = 256 / kWave;
        hipLaunchKernelGGL(sample_finish_kernel, dim3((p.B + wpb - 1) / wpb), dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace dspark
