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
//
// One workgroup counts a row in LDS and finds the drawn value there, then its index
// in the row. 2003 rows of 151936 (609 MB) take 160 us: reading them once and a half
// at 5.7 TB/s bounds that, with the LDS atomics (63 us) and vector instructions beside
// it. Two rows take 27 us: a CU's 1.5e5 atomics (8 us) and a chain of round trips. Rows
// that need the wide places take eight times as long (1259 us for all 2003). A row that
// holds a zero is read once more, two loads in flight, to tell zeros from values below
// 2^-32: all 2003 with 64 zeros each take 230 us, two 32 us.
#include "argmax_dev.hpp"
#include "forward.hpp"

namespace dspark {

constexpr int kSampleThreads = 512;
constexpr int kSampleWaves = kSampleThreads / kWave;
constexpr int kSampleWavesPerSimd = 6;  // three workgroups a CU
constexpr int kRowUnroll = 8;  // 16-byte loads in flight per lane
constexpr int kWideUnroll = 2;
constexpr int kListed = 1024;  // equals that are ranked by their indices

// Places. A value's place counts down the ranking; 256 places are a block, four
// to a lane, so that one ballot finds a block of the 49 narrow ones.
//
// Narrow places: |x| in [2^-32, 2^16), 128 values an octave and a sign, one
// place each, one more at either side of zero for what is smaller, and 64 at
// either end for what is larger, so that the lanes of a masked vocabulary do not
// meet at one. The counters of all of them take 49 KiB of LDS: three workgroups
// share a CU, and one's loads run beside another's atomics. A counter holds 16
// bits for each half of the row, so that the drawn entry is then looked for in
// its half only: HBM is read one and a half times. The end places and the two at
// zero hold more than one value, so a row is finished this way only if that does
// not matter: nothing at or above 2^16, nothing nonzero below 2^-32, what lies
// at or below -2^16 (masks, -inf) so far down that it weighs nothing
// (kNegligible), and no counter over 16 bits (the counts add up to V).
//
// Wide places: every bf16 value, 65536 places, counted in eight rounds over
// the row. Any row can be finished this way.
constexpr uint32_t kNarrowLo = (127 - 32) << 7, kNarrowHi = (127 + 16) << 7;  // bits of |x|
constexpr int kNarrowSpan = (int)(kNarrowHi - kNarrowLo);
constexpr int kPlaceZero = kWave + kNarrowSpan;  // +0 and what is below 2^-32
constexpr int kPlaceMinus = kPlaceZero + 1;      // -0 and what is above -2^-32
constexpr int kPlaceLow = kPlaceMinus + kNarrowSpan + 1;  // 64 places: -2^16 and below, NaN
constexpr uint32_t kFirstHalf = 1u, kSecondHalf = 1u << 16;
constexpr int kPer = 4;  // places of a lane
constexpr int kBlock = kPer * kWave;
constexpr int kNarrowBlocks = (kPlaceLow + kWave + kBlock - 1) / kBlock;
constexpr int kWideBlocks = 65536 / kBlock;
constexpr int kWideRound = 8192;  // counters of one round
// exp(-60) of the largest weight times 2^31 entries is 2e-17 of the sum, below
// the half step of the 64-bit sums.
constexpr double kNegligible = 60.0;

struct Narrow {
    static constexpr int kBlocks = kNarrowBlocks;
    uint32_t bins[kBlocks * kBlock];
    double wex[kBlocks + 1];  // weight and count before each block
    int cex[kBlocks + 1];
    __device__ static int count(uint32_t c) { return (int)((c & 0xFFFFu) + (c >> 16)); }
    // bits of the value at a place
    __device__ static uint32_t bits(int e) {
        e = e > kPlaceLow ? kPlaceLow : e;
        if (e == kPlaceZero || e == kPlaceMinus) return 0u;
        return e < kPlaceZero ? kNarrowHi - 1u - (uint32_t)(e - kWave)
                              : 0x8000u | (kNarrowLo - 1u + (uint32_t)(e - kPlaceMinus));
    }
};
struct Wide {
    static constexpr int kBlocks = kWideBlocks;
    __device__ static int count(uint32_t c) { return (int)c; }
    uint32_t bins[kWideRound];
    uint32_t detail[kBlock];  // counts of the block at hand
    double wex[kBlocks + 1];
    int cex[kBlocks + 1];
    __device__ static uint32_t bits(int e) {
        const uint32_t key = 0xFFFFu - (uint32_t)e;
        return key & 0x8000u ? key ^ 0x8000u : ~key & 0xFFFFu;
    }
};
struct alignas(16) SampleLds {
    union {
        Narrow narrow;
        Wide wide;
    };
    int part[kSampleWaves];
    int listed;    // entries found of the drawn value
    int counted;   // entries in the narrow places above kPlaceLow
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
    // vectors of the row's first half, where the head belongs too
    __device__ int half() const { return vecs / 2; }
    __device__ int loose() const { return V - 8 * vecs; }
    // index of the i-th entry outside the vectors
    __device__ int loose_at(int i) const { return i < head ? i : 8 * vecs + i; }
    __device__ const u32x4 *vec() const { return reinterpret_cast<const u32x4 *>(p + head); }
};

// f(vector, its number) for vectors [v0, v1), by lanes `step` apart, the first
// of them at v0 + lane; f must take lanes that are off.
template <int kUnroll = kRowUnroll, typename F>
__device__ __forceinline__ void for_vecs(const Row &row, int v0, int v1, int lane, int step, F f) {
    const u32x4 *at = row.vec();
    int v = v0 + lane;
    for (; v + (kUnroll - 1) * step < v1; v += kUnroll * step) {
        u32x4 a[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) a[i] = at[v + i * step];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) f(a[i], v + i * step);
    }
    if (v < v1) {  // the last round's loads past the end repeat its first
        u32x4 a[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) a[i] = at[v + i * step < v1 ? v + i * step : v];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (v + i * step < v1) f(a[i], v + i * step);
    }
}
// f(bits) for every entry of the row, by the whole workgroup.
template <typename F>
__device__ __forceinline__ void for_row(const Row &row, F f) {
    for_vecs<kWideUnroll>(row, 0, row.vecs, threadIdx.x, kSampleThreads, [&](u32x4 a, int) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f(a[i] & 0xFFFFu);
            f(a[i] >> 16);
        }
    });
    if ((int)threadIdx.x < row.loose()) f((uint32_t)row.p[row.loose_at(threadIdx.x)]);
}

// Byte offsets of the counters of two values' narrow places, packed: seven
// instructions for two values (a 16-bit shift of both signs at once is not
// found by the compiler). `end` is the lane's distance to its end places.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 narrow_end() {
    const unsigned short e = (unsigned short)(kNarrowSpan + 1 + (threadIdx.x & (kWave - 1)));
    return u16x2{e, e};
}
__device__ __forceinline__ uint32_t narrow_offsets(uint32_t two, u16x2 end) {
    constexpr unsigned short lo = kNarrowLo - 1, c = 4 * kPlaceMinus;
    u16x2 m = __builtin_bit_cast(u16x2, two & 0x7FFF7FFFu);
    m = __builtin_elementwise_min(__builtin_elementwise_sub_sat(m, (u16x2){lo, lo}),
                                  end);
    // the place is kPlaceZero - m for a positive value, kPlaceMinus + m for a negative one
    uint32_t sign;
    asm("v_pk_ashrrev_i16 %0, 15, %1 op_sel_hi:[0,1]" : "=v"(sign) : "v"(two));
    const u16x2 e = __builtin_bit_cast(u16x2, ~(__builtin_bit_cast(uint32_t, m) ^ sign));
    return __builtin_bit_cast(uint32_t, (u16x2)(e * (u16x2){4, 4} + (u16x2){c, c}));
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
    double T, per_T, u, top_p, min_p;  // per_T = 1 / T
    int k;
};
// What a row draws: the bits of its value, which of its equals, and its place.
struct Drawn {
    uint32_t bits;
    int j, place;
};

// Counts and weights of all blocks are in place (prefix sums in wex and cex,
// totals at their ends); every wave walks the filters by itself, with the
// same numbers. counts(t) gives lane l the counts of places kBlock*t + kPer*l on.
template <typename H, typename Weight, typename Counts>
__device__ __forceinline__ Drawn walk_filters(const H &h, const Draw &d, Weight weight,
                                              Counts counts) {
    const int lane = threadIdx.x & (kWave - 1);
    // the first block for which `test` holds, -1 if none
    auto first = [&](auto test) {
#pragma unroll 1
        for (int i0 = 0; i0 < H::kBlocks; i0 += kWave) {
            const int i = i0 + lane;
            const uint64_t m = __ballot(i < H::kBlocks && test(i));
            if (m) return i0 + __ffsll((unsigned long long)m) - 1;
        }
        return -1;
    };
    // counts and weights of this lane's places in block t, and what precedes them
    int n[kPer] = {}, before[kPer] = {}, have = -1;
    double w[kPer] = {}, ahead[kPer] = {};
    auto open = [&](int t) {
        if (t == have) return;
        have = t;
        const u32x4 c = counts(t);
        int sum = 0;
        double x = 0.0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            n[u] = H::count(c[u]);
            w[u] = n[u] ? weight(t * kBlock + kPer * lane + u) : 0.0;
            before[u] = sum;
            ahead[u] = x;
            sum += n[u];
            x += (double)n[u] * w[u];
        }
        const int b0 = h.cex[t] + wave_incl_scan(sum, lane) - sum;
        const double a0 = h.wex[t] + (wave_incl_sum(x) - x);
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            before[u] += b0;
            ahead[u] += a0;
        }
    };
    auto wave_sum = [&](int x) { return last_lane(wave_incl_scan(x, lane)); };
    int N = h.cex[H::kBlocks];
    double total = h.wex[H::kBlocks];
    auto cut = [&](int keep) {
        keep = keep < 1 ? 1 : keep;
        if (keep >= N) return;
        const int t = first([&](int i) { return h.cex[i + 1] >= keep; });
        open(t);
        double x = 0.0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            int mine = keep - before[u];
            mine = mine < 0 ? 0 : (mine > n[u] ? n[u] : mine);
            x += (double)mine * w[u];
        }
        total = h.wex[t] + last_lane(wave_incl_sum(x));
        N = keep;
    };
    // Entries of the open block that come before `goal`: of a place the first m
    // with ahead + (m - 1) w below it or, `whole`, with ahead + m w at most it.
    // One place at most holds the border; only there m is searched for.
    auto entries = [&](double goal, bool whole) {
        auto in = [&](double a, double x, int m) {
            return whole ? a + (double)m * x <= goal : a + (double)(m - 1) * x < goal;
        };
        int sum = 0, c = 0;
        double a = 0.0, x = 0.0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            if (n[u] == 0 || !in(ahead[u], w[u], 1)) continue;
            if (in(ahead[u], w[u], n[u])) {
                sum += n[u];
            } else {
                c = n[u];
                a = ahead[u];
                x = w[u];
            }
        }
        if (c) {
            const double q = (goal - a) / x;
            int m = q < 1.0 ? 1 : (q < (double)c ? (int)q : c);
            while (m > 1 && !in(a, x, m)) --m;
            while (m < c && in(a, x, m + 1)) ++m;
            sum += m;
        }
        return wave_sum(sum);
    };
    if (d.k > 0) cut(d.k);
    if (d.top_p < 1.0) {
        const double goal = d.top_p * total;
        const int t = goal > 0.0 ? first([&](int i) {
            return h.cex[i + 1] > h.cex[i] && !(h.wex[i + 1] < goal);
        }) : -1;
        if (t >= 0) {
            open(t);
            cut(h.cex[t] + entries(goal, false));
        } else if (!(goal > 0.0)) {
            cut(1);
        }
    }
    if (d.min_p > 0.0) {
        // the first block that is not kept whole
        const int t = first([&](int i) {
            return h.cex[i + 1] > h.cex[i] && !(weight(i * kBlock + kBlock - 1) >= d.min_p);
        });
        if (t >= 0) {
            open(t);
            int m = 0;
#pragma unroll
            for (int u = 0; u < kPer; ++u) m += n[u] && w[u] >= d.min_p ? n[u] : 0;
            cut(h.cex[t] + wave_sum(m));
        }
    }
    const double goal = d.u * total;
    int rank = N - 1;
    const int t = first([&](int i) {
        return h.cex[i + 1] > h.cex[i] && !(h.wex[i + 1] <= goal);
    });
    if (t >= 0) {
        open(t);
        const int x = h.cex[t] + entries(goal, true);
        rank = x < rank ? x : rank;
    }
    const int at = first([&](int i) { return h.cex[i + 1] > rank; });
    open(at);
    int place = 0, nth = 0;
    bool mine = false;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        if (before[u] <= rank && rank < before[u] + n[u]) {
            mine = true;
            place = at * kBlock + kPer * lane + u;
            nth = rank - before[u];
        }
    }
    const int l = __ffsll((unsigned long long)__ballot(mine)) - 1;
    Drawn r;
    r.place = __builtin_amdgcn_readlane(place, l);
    r.bits = H::bits(r.place);
    r.j = __builtin_amdgcn_readlane(nth, l);
    return r;
}

// Count and weight of block i from its counters; a lane's four exponentials run
// side by side.
template <typename H, typename Weight>
__device__ __forceinline__ void sum_block(H &h, int i, const uint32_t *bins, Weight weight) {
    const int lane = threadIdx.x & (kWave - 1);
    const u32x4 n = reinterpret_cast<const u32x4 *>(bins)[lane];
    int c = 0;
    double w = 0.0;
    if (__ballot((n[0] | n[1] | n[2] | n[3]) != 0)) {
        double x[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) x[u] = weight(i * kBlock + kPer * lane + u);
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int k = H::count(n[u]);
            c += k;
            w += k ? (double)k * x[u] : 0.0;
        }
        c = last_lane(wave_incl_scan(c, lane));
        w = last_lane(wave_incl_sum(w));
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
#pragma unroll 1
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

// Which entries equal a value (zeros of either sign are equal: kZero).
template <bool kZero>
struct Equal {
    static constexpr uint32_t kMask = kZero ? 0x7FFF7FFFu : 0xFFFFFFFFu;
    uint32_t want;
    __device__ explicit Equal(uint32_t bits) : want(bits | (bits << 16)) {}
    __device__ __forceinline__ bool one(uint32_t x) const {
        return ((x ^ want) & kMask & 0xFFFFu) == 0;
    }
    // a bit per entry of a vector; the usual one holds none, which the smallest
    // of the eight differences shows
    __device__ __forceinline__ uint32_t vec(u32x4 a) const {
        uint32_t t[4];
        u16x2 least = {0xFFFF, 0xFFFF};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = (a[i] ^ want) & kMask;
            least = __builtin_elementwise_min(least, __builtin_bit_cast(u16x2, t[i]));
        }
        uint32_t m = 0;
        if (least[0] == 0 || least[1] == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m |= ((t[i] & 0xFFFFu) == 0 ? 1u << (2 * i) : 0u) |
                     (t[i] >> 16 == 0 ? 2u << (2 * i) : 0u);
        }
        return m;
    }
};

// The vectors of wave w: a contiguous share, in steps of a wave.
struct Share {
    int v0, v1;
    __device__ Share(const Row &row, int w) {
        const int per = (row.vecs + kSampleWaves * kWave - 1) / (kSampleWaves * kWave) * kWave;
        v0 = w * per < row.vecs ? w * per : row.vecs;
        v1 = v0 + per < row.vecs ? v0 + per : row.vecs;
    }
};

// The index of the (j+1)-th of the row's entries that equal the drawn value, by
// reading the row again.
template <bool kZero>
__device__ __forceinline__ int index_of(SampleLds &s, const Row &row, const Drawn &d) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const Equal<kZero> equal(d.bits);
    const bool edge = tid < row.loose() && equal.one(row.p[row.loose_at(tid)]);
    const Share mine(row, wave);
    int c = 0;
    for_vecs(row, mine.v0, mine.v1, lane, kWave,
             [&](u32x4 a, int) { c += __popc(equal.vec(a)); });
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
        for (int v = mine.v0; v < mine.v1; v += kWave) {
            const uint32_t m = v + lane < mine.v1 ? equal.vec(row.vec()[v + lane]) : 0u;
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

// index_of among the row's entries of one half, up to kListed equals: all of
// them are listed, and the one with j smaller indices is taken.
template <bool kZero>
__device__ __forceinline__ int index_in_half(SampleLds &s, const Row &row, bool second,
                                             const Drawn &d) {
    const int tid = threadIdx.x;
    const Equal<kZero> equal(d.bits);
    int *list = reinterpret_cast<int *>(s.narrow.bins);
    auto found = [&](int i) {
        const int slot = atomicAdd(&s.listed, 1);
        if (slot < kListed) list[slot] = i;
    };
    if (tid < row.loose() && (tid >= row.head) == second && equal.one(row.p[row.loose_at(tid)]))
        found(row.loose_at(tid));
    for_vecs(row, second ? row.half() : 0, second ? row.vecs : row.half(), tid, kSampleThreads,
             [&](u32x4 a, int v) {
                 for (uint32_t m = equal.vec(a); m; m &= m - 1)
                     found(row.head + 8 * v + __ffs((int)m) - 1);
             });
    __syncthreads();
    const int n = s.listed < kListed ? s.listed : kListed;
    for (int i = tid; i < n; i += kSampleThreads) {
        const int x = list[i];
        int before = 0;
        for (int k = 0; k < n; ++k) before += list[k] < x;
        if (before == d.j) s.at = x;
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
    if (!(d.T > 0.0) || d.k == 1) return Drawn{Wide::bits(first), 0, 0};
    const double vmax = (double)bf16_f32((uint16_t)Wide::bits(first));
    auto weight = [&](int e) {
        return e == first ? 1.0 : exp(((double)bf16_f32((uint16_t)Wide::bits(e)) - vmax) * d.per_T);
    };
#pragma unroll 1
    for (int round = 0; round < 65536 / kWideRound; ++round) {
        for (int i = tid; i < kWideRound; i += kSampleThreads) h.bins[i] = 0;
        __syncthreads();
        for_row(row, [&](uint32_t x) {
            const uint32_t key = value_key(x), e = 0xFFFFu - key;
            if (key_counts(key) && (int)(e / kWideRound) == round)
                atomicAdd(&h.bins[e % kWideRound], 1u);
        });
        __syncthreads();
#pragma unroll 1
        for (int i = wave; i < kWideRound / kBlock; i += kSampleWaves)
            sum_block(h, round * (kWideRound / kBlock) + i, h.bins + i * kBlock, weight);
        __syncthreads();
    }
    if (wave == 0) scan_blocks(h);
    __syncthreads();
    return walk_filters(h, d, weight, [&](int t) {
        __syncthreads();
        if (tid < kBlock) h.detail[tid] = 0;
        __syncthreads();
        for_row(row, [&](uint32_t x) {
            const uint32_t key = value_key(x), e = 0xFFFFu - key;
            if (key_counts(key) && (int)(e / kBlock) == t) atomicAdd(&h.detail[e % kBlock], 1u);
        });
        __syncthreads();
        return reinterpret_cast<const u32x4 *>(h.detail)[lane];
    });
}

// The request that owns packed row r: the first whose end lies past it (B if
// none does), so that rows have one owner each whatever cu holds. `below` is this
// lane's largest end of an earlier request: the wave's largest is where the
// owner's rows start.
__device__ __forceinline__ int wave_owner_of(const int32_t *__restrict__ cu, int B, int r,
                                             int &below) {
    const int lane = threadIdx.x & (kWave - 1);
    below = 0;
    for (int i0 = 0; i0 < B; i0 += 4 * kWave) {
        int x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kWave + lane;
            x[u] = i < B ? cu[i + 1] : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint64_t m = __ballot(x[u] > r);
            const int first = m ? __ffsll((unsigned long long)m) - 1 : kWave;
            if (lane < first && x[u] > below) below = x[u];
            if (m) return i0 + u * kWave + first;
        }
    }
    return B;
}
__device__ __forceinline__ int wave_max_int(int x) {
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) {
        const int y = __shfl_xor(x, off, kWave);
        x = y > x ? y : x;
    }
    return x;
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
    // accepted and bonus of request r, if it has no rows; by one wave
    auto settle_empty = [&]() {
        int start = 0;
        for (int i = lane; i <= r; i += kWave) start = p.cu[i] > start ? p.cu[i] : start;
        start = wave_max_int(start);
        if (lane == 0 && (p.cu[r + 1] <= start || start >= total)) {
            p.acc[r] = 0;
            p.bonus[r] = -1;
        }
    };
    if (r >= total) {
        if (arrivals && r < p.B && wave == 0) settle_empty();
        return;
    }
    const bool exists = src >= 0 && src < cap;
    const Row row(p.logits + (int64_t)(exists ? src : 0) * p.V, exists ? p.V : 0);
    int below;
    const int b = wave_owner_of(p.cu, p.B, r, below);
    Draw d;
    const bool owned = b < p.B && r >= p.cu[0];
    d.T = owned && p.temperature ? (double)p.temperature[b] : 1.0;
    d.k = owned && p.top_k ? p.top_k[b] : 0;
    d.top_p = owned && p.top_p ? (double)p.top_p[b] : 1.0;
    d.min_p = owned && p.min_p ? (double)p.min_p[b] : 0.0;
    d.u = p.uniforms[r] > 0.f ? (double)p.uniforms[r] : 0.0;
    for (int i = tid; i < kNarrowBlocks * kBlock / 4; i += kSampleThreads)
        reinterpret_cast<u32x4 *>(h.bins)[i] = u32x4{0u, 0u, 0u, 0u};
    if (tid == 0) {
        s.top = kNarrowBlocks * kBlock;
        s.flag = 0;
        s.listed = 0;
        s.counted = 0;
    }
    __syncthreads();
    {
        char *bins = reinterpret_cast<char *>(h.bins);
        const u16x2 end = narrow_end();
        auto add = [&](uint32_t off, uint32_t one) {
            atomicAdd(reinterpret_cast<uint32_t *>(bins + off), one);
        };
        auto count = [&](int v0, int v1, uint32_t one) {
            for_vecs(row, v0, v1, tid, kSampleThreads, [&](u32x4 a, int) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = narrow_offsets(a[i], end);
                    add(two & 0xFFFFu, one);
                    add(two >> 16, one);
                }
            });
        };
        count(0, row.half(), kFirstHalf);
        count(row.half(), row.vecs, kSecondHalf);
        if (tid < row.loose())
            add(narrow_offsets(row.p[row.loose_at(tid)], end) & 0xFFFFu,
                tid < row.head ? kFirstHalf : kSecondHalf);
    }
    __syncthreads();

    d.per_T = 1.0 / d.T;
    const bool high = __ballot(h.bins[lane] != 0) != 0;
    const int low = last_lane(wave_incl_scan(Narrow::count(h.bins[kPlaceLow + lane]), lane));
    const uint32_t z0 = h.bins[kPlaceZero], z1 = h.bins[kPlaceMinus];
    const uint32_t zeros[2] = {(z0 & 0xFFFFu) + (z1 & 0xFFFFu), (z0 >> 16) + (z1 >> 16)};
    if (zeros[0] | zeros[1]) {  // is it only zeros, and do they fit?
        bool small = (zeros[0] | zeros[1]) > 0xFFFFu;
        for_row(row, [&](uint32_t x) {
            const uint32_t m = x & 0x7FFFu;
            small |= m > 0 && m < kNarrowLo;
        });
        if (small) s.flag = 1;
    }
    __syncthreads();
    if (wave == 0) h.bins[kPlaceLow + lane] = 0;
    if (tid == 0) {
        h.bins[kPlaceZero] = zeros[0] | zeros[1] << 16;
        h.bins[kPlaceMinus] = 0;
    }
    __syncthreads();
    int sum = 0;
    bool empty = true;
#pragma unroll 1
    for (int i = wave; i < kNarrowBlocks; i += kSampleWaves) {
        const u32x4 n = reinterpret_cast<const u32x4 *>(h.bins + i * kBlock)[lane];
        const uint64_t m = __ballot((n[0] | n[1] | n[2] | n[3]) != 0);
        if (m == 0) continue;
        if (empty && lane == __ffsll((unsigned long long)m) - 1)
            atomicMin(&s.top, (unsigned)(i * kBlock + kPer * lane +
                                         (n[0] ? 0 : n[1] ? 1 : n[2] ? 2 : 3)));
        empty = false;
#pragma unroll
        for (int u = 0; u < kPer; ++u) sum += Narrow::count(n[u]);
    }
    sum = last_lane(wave_incl_scan(sum, lane));
    if (lane == 0) atomicAdd(&s.counted, sum);
    __syncthreads();
    const int top = (int)s.top;
    const bool small = s.flag != 0;
    const bool greedy = !(d.T > 0.0) || d.k == 1;
    const double vmax = (double)bf16_f32((uint16_t)Narrow::bits(top));
    const bool narrow = !high && !small && top < kPlaceLow && s.counted + low == row.V &&
                  (low == 0 || greedy || (vmax + 65536.0) * d.per_T > kNegligible);
    Drawn out;
    if (narrow && greedy) {
        out = Drawn{Narrow::bits(top), 0, top};
    } else if (narrow) {
        auto weight = [&](int e) {
            return exp(((double)bf16_f32((uint16_t)Narrow::bits(e)) - vmax) * d.per_T);
        };
#pragma unroll 1
        for (int i = wave; i < kNarrowBlocks; i += kSampleWaves)
            sum_block(h, i, h.bins + i * kBlock, weight);
        __syncthreads();
        if (wave == 0) scan_blocks(h);
        __syncthreads();
        out = walk_filters(h, d, weight, [&](int t) {
            return reinterpret_cast<const u32x4 *>(h.bins + t * kBlock)[lane];
        });
    }
    int chosen = -1;
    if (exists && narrow) {
        const uint32_t c = h.bins[out.place];
        const int ahead = (int)(c & 0xFFFFu), all = Narrow::count(c);
        const bool second = out.j >= ahead;
        __syncthreads();
        if ((second ? all - ahead : ahead) <= kListed) {
            Drawn in = out;
            in.j -= second ? ahead : 0;
            chosen = out.bits ? index_in_half<false>(s, row, second, in)
                              : index_in_half<true>(s, row, second, in);
        } else {
            chosen = out.bits ? index_of<false>(s, row, out) : index_of<true>(s, row, out);
        }
    } else if (exists) {
        __syncthreads();
        out = draw_wide(s, row, d);
        // nothing to draw from: the lowest index
        if (out.j < 0) chosen = 0;
        else chosen = out.bits ? index_of<false>(s, row, out) : index_of<true>(s, row, out);
    }
    if (arrivals && r < p.B && wave == 1) settle_empty();
    if (!owned || wave != 0) return;
    if (!arrivals) {
        if (lane == 0) p.sample[r] = chosen;
        return;
    }
    // the last row of a request to arrive accepts its drafts
    below = below > p.cu[0] ? below : p.cu[0];
    const int start = wave_max_int(below);
    const int end = p.cu[b + 1] < total ? p.cu[b + 1] : total, n = end - start;
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
