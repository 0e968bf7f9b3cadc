// attend.hip - attention of the packed verify rows over each request's pages of
// the key-value cache.
//
// Row j of request b stands at position p = ctx[b] + j and sees the positions
// max(0, p - window + 1) .. p (from 0 without a window) whose page the table
// names:
//   O = sum_t exp(x_t - m) V_t / sum_t exp(x_t - m),  x_t = scale (q . K_t),
// with m the largest x_t. A running maximum and sum carry the softmax over the
// keys in one pass; a row that sees nothing gives zeros.
#include "forward.hpp"

namespace dspark {

constexpr int kMaxHeadDim = 256;
constexpr int kRowThreads = 64;

template <bool kE4m3>
__device__ __forceinline__ void load8(const void *pool, int64_t at, float *x) {
    if (kE4m3) {
        const uint64_t w =
            *reinterpret_cast<const uint64_t *>(static_cast<const uint8_t *>(pool) + at);
        const int lo = (int)(uint32_t)w, hi = (int)(uint32_t)(w >> 32);
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(lo, false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(lo, true);
        const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(hi, false);
        const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8(hi, true);
        x[0] = a[0]; x[1] = a[1]; x[2] = b[0]; x[3] = b[1];
        x[4] = c[0]; x[5] = c[1]; x[6] = d[0]; x[7] = d[1];
    } else {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(pool) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}
template <bool kE4m3>
__device__ __forceinline__ float load1(const void *pool, int64_t at) {
    if (kE4m3)
        return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t *>(pool)[at], 0);
    return bf16_f32(static_cast<const uint16_t *>(pool)[at]);
}

// One wave per (packed row, query head): 64 keys at a time, a lane per key for
// the scores and a lane per output element for the weighted values.
template <bool kE4m3>
__global__ __launch_bounds__(kRowThreads) void attend_row_kernel(AttendParams p) {
    __shared__ float q_s[kMaxHeadDim];
    __shared__ float p_s[kWave];
    __shared__ int64_t at_s[kWave];
    const int lane = threadIdx.x;
    const int r = blockIdx.x, h = blockIdx.y;
    const int b = wave_request_of(p.cu, p.B, r);
    if (b >= p.B) return;
    const int j = r - p.cu[b];
    if (j < 0 || j >= p.max_rows) return;
    const int kvh = h / (p.Hq / p.Hkv);
    // positions past the table's width have no page
    const int64_t width = (int64_t)p.c.table_width * p.c.page;
    const int64_t pos = (int64_t)(p.ctx[b] < 0 ? 0 : p.ctx[b]) + j;
    const int64_t end = pos + 1 < width ? pos + 1 : width;
    const int64_t begin = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    const int32_t *row = p.c.table + (int64_t)b * p.c.table_width;
    const uint16_t *q = p.q + r * p.q_row + h * p.q_head;
    for (int d = lane; d < p.D; d += kWave) q_s[d] = bf16_f32(q[d]) * p.scale * p.c.k_scale;
    __syncthreads();
    float m = -INFINITY, total = 0.f;
    float acc[kMaxHeadDim / kWave] = {};
    for (int64_t t0 = begin; t0 < end; t0 += kWave) {
        const int64_t t = t0 + lane;
        const int64_t at = t < end ? slot_offset(p.c, row, (int)t, kvh) : -1;
        float x = -INFINITY;
        if (at >= 0) {
            x = 0.f;
            for (int d = 0; d < p.D; d += 8) {
                float k[8];
                load8<kE4m3>(p.c.k, at + d, k);
#pragma unroll
                for (int i = 0; i < 8; ++i) x += q_s[d + i] * k[i];
            }
        }
        float top = x;
#pragma unroll
        for (int off = kWave / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
        const float m1 = fmaxf(m, top);
        if (m1 == -INFINITY) continue;
        const float keep = expf(m - m1);
        const float w = at >= 0 ? expf(x - m1) : 0.f;
        m = m1;
        total = total * keep + wave_sum_f32(w);
        p_s[lane] = w;
        at_s[lane] = at;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMaxHeadDim / kWave; ++i) {
            const int d = i * kWave + lane;
            if (d < p.D) {
                float a = acc[i] * keep;
                for (int u = 0; u < kWave; ++u)
                    if (at_s[u] >= 0) a += p_s[u] * load1<kE4m3>(p.c.v, at_s[u] + d);
                acc[i] = a;
            }
        }
        __syncthreads();
    }
    uint16_t *o = p.out + ((int64_t)r * p.Hq + h) * p.D;
    const float norm = total > 0.f ? p.c.v_scale / total : 0.f;
#pragma unroll
    for (int i = 0; i < kMaxHeadDim / kWave; ++i) {
        const int d = i * kWave + lane;
        if (d < p.D) o[d] = (uint16_t)pack_bf16(acc[i] * norm, 0.f);
    }
}

// ---------------------------------------------------------------- tiled kernel
//
// Rows of one key-value head share its keys: with G query heads per key-value
// head, a request's n rows are M = n*G query rows, taken in blocks of up to 128
// against tiles of 64 positions. A (head, block) is a unit; the tiles of all units,
// laid end to end, are divided evenly between the resident workgroups, so any
// mix of long and short requests fills the chip, a single long context
// included, and no launch shape depends on the lengths. A unit that ends up in
// several workgroups leaves partial results (maximum, sum, weighted values) in
// the workspace, and the last workgroup to arrive joins them in tile order.
//
// Scores are computed transposed, S^T = K Q^T: a lane then holds 16 of a query's 32
// scores of one MFMA (the other 16 sit in lane ^ 32), so the softmax needs one
// exchange between the halves, and the weights leave the exponential in the
// very places where the next product, O^T = V^T P^T, wants them. V^T comes
// from row-major V in LDS through the transposing LDS reads.
//
// Weights are rounded to bf16 before their product with V (half a step 2^-8 of
// each weight, averaged over the keys); sums, maxima and outputs stay in fp32.

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kTileKeys = 64;
constexpr int kBlockRows = 128;
constexpr int kTileThreads = 256;
constexpr int kTileWaves = kTileThreads / kWave;
constexpr int kTileWgsPerCu = 2;
constexpr int kGroupRequests = 1024;  // of one launch; larger batches take several
constexpr int kMinTiles = 2;          // per workgroup: fewer would cost more to join than to read
constexpr float kLog2e = 1.44269504088896340736f;

struct TileParams {
    AttendParams a;
    unsigned *arrivals;  // [wgs], zero between calls
    float *slots;        // [2 * wgs] partial results of slot_rows rows
    int slot_rows;
};

// Floats of one partial result: (maximum, sum) and D values of each row.
__host__ __device__ inline int64_t slot_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

struct Request {
    int start, ctx, M, blocks;
};
__device__ __forceinline__ Request load_request(const AttendParams &p, int b) {
    Request q;
    int s = p.cu[b], e = p.cu[b + 1];
    s = s < 0 ? 0 : (s > p.rows ? p.rows : s);
    e = e < s ? s : (e > p.rows ? p.rows : e);
    const int n = e - s < p.max_rows ? e - s : p.max_rows;
    const int c = p.ctx[b];
    q.start = s;
    q.ctx = c < 0 ? 0 : (c > (1 << 30) ? 1 << 30 : c);
    q.M = n * (p.Hq / p.Hkv);
    q.blocks = (q.M + kBlockRows - 1) / kBlockRows;
    return q;
}
// Positions [lo, hi) that block i of a request needs, and its tiles (one at
// least: a block that sees nothing still writes its zeros).
struct Block {
    int lo, hi, tile, tiles;
};
__device__ __forceinline__ Block block_of(const AttendParams &p, const Request &q, int i) {
    const int G = p.Hq / p.Hkv;
    const int m0 = i * kBlockRows;
    const int m1 = (q.M < m0 + kBlockRows ? q.M : m0 + kBlockRows) - 1;
    const int64_t width = (int64_t)p.c.table_width * p.c.page;
    Block k;
    k.lo = 0;
    if (p.window > 0 && q.ctx + m0 / G + 1 > p.window) k.lo = q.ctx + m0 / G + 1 - p.window;
    const int end = q.ctx + m1 / G + 1;
    k.hi = end < width ? end : (int)width;
    k.tile = k.lo / kTileKeys;
    const int last = (k.hi + kTileKeys - 1) / kTileKeys;
    k.tiles = last > k.tile ? last - k.tile : 1;
    return k;
}

__device__ __forceinline__ uint64_t wave_incl_sum_u64(uint64_t x) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const uint64_t y = __shfl_up(x, off, kWave);
        if (lane >= off) x += y;
    }
    return x;
}

// The value of the other half's lane (lane ^ 32) combined with the own one.
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ void store_coherent(float *p, float a, float b) {
    const uint64_t v = (uint64_t)__float_as_uint(a) | ((uint64_t)__float_as_uint(b) << 32);
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), v, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x2 load_coherent(const float *p) {
    const uint64_t v = __hip_atomic_load(reinterpret_cast<uint64_t *>(const_cast<float *>(p)),
                                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return f32x2{__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))};
}

// Chunk (16 bytes) c of row r of a staged tile sits at chunk c ^ swizzle(r): 16
// neighbouring rows then lie in different banks for the score operand (one
// chunk of 32 rows), and 4 rows in different quarters of the banks for the
// transposed reads (4 chunks of 8 rows).
template <int D>
__device__ __forceinline__ int swizzle(int r) {
    if (D >= 128) return ((r & 3) << 2) | ((r >> 2) & 3);
    return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

template <int D, bool kE4m3>
struct Tiles {
    static constexpr int kItem = kE4m3 ? 1 : 2;
    static constexpr int kRowLanes = D * kItem / 16;       // lanes of 16 bytes per row
    static constexpr int kLoadRows = kWave / kRowLanes;    // rows of one wave's load
    static constexpr int kLoads = 16 / kLoadRows;          // a wave stages 16 rows of a tile
    static constexpr int kTileBytes = kTileKeys * D * 2;   // of K or V in LDS, as bf16

    struct Lds {
        union {
            char stage[2][2][kTileBytes];  // [buffer][K, V]
            float join[2][(D / 2 + 2) * kWave];
        };
        uint64_t before[kGroupRequests + 1];
        uint64_t part[kTileWaves];
        // a bit per row of a wave's 16: those without a page, and in the upper
        // half those whose values were not all finite
        uint32_t marks[2][kTileWaves];
        int last;
    };

    // What one wave works on inside a unit.
    struct Task {
        const int32_t *table;
        int64_t head_off;   // of the key-value head in the pools
        int lo, hi;         // positions that exist for the block
        int ctx, pos;       // of the request; of this lane's query row
        int pos_min, pos_max;  // over the wave's query rows
        int first, final;      // over the block's
        bool active;
        float c;            // scores to powers of two
    };
    struct State {
        bf16x8 q[D / 16];
        f32x16 o[D / 32];
        float m, l;
    };
    struct Regs {
        u32x4 k[kLoads], v[kLoads];
        int holes;
    };
    struct Entry {
        int at[kLoads];
    };

    __device__ static __forceinline__ int wave_id() {
        return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    }

    // Table entries of the rows that this lane loads of a tile (-1: no page).
    // Pages of a multiple of 16 slots hold a wave's 16 rows together.
    __device__ static __forceinline__ void lookup(const PagedCache &c, const Task &t, int tile,
                                                  Entry &e) {
        const int lane = threadIdx.x & (kWave - 1);
        const int first = tile * kTileKeys + wave_id() * 16;
        if (c.page % 16 == 0) {
            const int pg = page_of(c, first);
            e.at[0] = pg < c.table_width ? t.table[pg] : -1;
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int pg = page_of(c, first + i * kLoadRows + lane / kRowLanes);
                e.at[i] = pg < c.table_width ? t.table[pg] : -1;
            }
        }
    }
    __device__ static __forceinline__ void load(const PagedCache &c, const Task &t, int tile,
                                                const Entry &e, Regs &g) {
        const int lane = threadIdx.x & (kWave - 1);
        const int first = tile * kTileKeys + wave_id() * 16;
        const bool together = c.page % 16 == 0;
        const char *kp = static_cast<const char *>(c.k), *vp = static_cast<const char *>(c.v);
        g.holes = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = i * kLoadRows + lane / kRowLanes;
            const int pos = first + r;
            const int at = together ? e.at[0] : e.at[i];
            const int pg = together ? page_of(c, first) : page_of(c, pos);
            const bool named = at >= 0 && at < c.pages;
            const bool here = named && pos >= t.lo && pos < t.hi;
            // one bit per row: lanes of the row's first chunk
            const uint64_t no = __ballot(!named);
#pragma unroll
            for (int x = 0; x < kLoadRows; ++x)
                g.holes |= (int)(no >> (x * kRowLanes) & 1) << (i * kLoadRows + x);
            g.k[i] = u32x4{0u, 0u, 0u, 0u};
            g.v[i] = u32x4{0u, 0u, 0u, 0u};
            if (here) {
                const int64_t off =
                    ((int64_t)at * c.page_stride + (int64_t)(pos - pg * c.page) * c.slot_stride +
                     t.head_off) * kItem + (lane % kRowLanes) * 16;
                g.k[i] = *reinterpret_cast<const u32x4 *>(kp + off);
                g.v[i] = *reinterpret_cast<const u32x4 *>(vp + off);
            }
        }
    }
    __device__ static __forceinline__ u32x4 widen(uint32_t a, uint32_t b) {
        return u32x4{
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true))};
    }
    __device__ static __forceinline__ void put(char *buf, int r, int lane, u32x4 x, bool scrub,
                                               bool &bad) {
        const int f = swizzle<D>(r), c = lane % kRowLanes;
        char *row = buf + r * (D * 2);
        if (kE4m3) {  // 16 values are two chunks of bf16, exactly
            u32x4 y = widen(x[0], x[1]), z = widen(x[2], x[3]);
            if (scrub) bad = scrubbed(y) | scrubbed(z);
            *reinterpret_cast<u32x4 *>(row + (((2 * c) ^ f) << 4)) = y;
            *reinterpret_cast<u32x4 *>(row + (((2 * c + 1) ^ f) << 4)) = z;
        } else {
            if (scrub) bad = scrubbed(x);
            *reinterpret_cast<u32x4 *>(row + ((c ^ f) << 4)) = x;
        }
    }
    // Sets what is not finite to 0; whether anything was.
    __device__ static __forceinline__ bool scrubbed(u32x4 &x) {
        u16x2 top = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x[i] & 0x7F807F80u));
        const bool bad = top[0] == 0x7F80 || top[1] == 0x7F80;
        if (bad) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if ((x[i] & 0x7F80u) == 0x7F80u) x[i] &= 0xFFFF0000u;
                if ((x[i] & 0x7F800000u) == 0x7F800000u) x[i] &= 0xFFFFu;
            }
        }
        return bad;
    }
    // Whether some row of the block does not see some key of the tile that another
    // one sees. There a weight of zero must keep out whatever the value is, which
    // zero times an infinity or NaN would not: values that are not finite are
    // staged as 0, and add_bad adds them to the rows that see them.
    __device__ static __forceinline__ bool partial(const AttendParams &p, const Task &t, int tile) {
        const int k0 = tile * kTileKeys;
        return k0 + kTileKeys - 1 > t.first || (p.window > 0 && k0 <= t.final - p.window);
    }
    __device__ static __forceinline__ void store(Lds &s, int buf, const Regs &g, bool scrub) {
        const int lane = threadIdx.x & (kWave - 1);
        uint32_t marks = (uint32_t)g.holes;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = wave_id() * 16 + i * kLoadRows + lane / kRowLanes;
            bool bad = false;
            put(s.stage[buf][0], r, lane, g.k[i], false, bad);
            put(s.stage[buf][1], r, lane, g.v[i], scrub, bad);
            const uint64_t m = __ballot(bad);
            if (m) {
#pragma unroll
                for (int x = 0; x < kLoadRows; ++x)
                    marks |= (m >> (x * kRowLanes) & ((1ull << kRowLanes) - 1))
                                 ? 0x10000u << (i * kLoadRows + x) : 0u;
            }
        }
        if (lane == 0) s.marks[buf][wave_id()] = marks;
    }

    // The values that `store` left out, from the cache again: to the rows that
    // see them. Their weights do not matter: the sum is not finite with any.
    __device__ static __forceinline__ void add_bad(const uint32_t *marks, int tile, int sub,
                                                   int keys, const AttendParams &p, const Task &t,
                                                   State &st) {
        const int h = (threadIdx.x >> 5) & 1;
#pragma unroll 1
        for (int y = sub * 32; y < sub * 32 + keys; ++y) {
            if (!(marks[y / 16] >> (16 + y % 16) & 1)) continue;
            const int key = tile * kTileKeys + y, pg = page_of(p.c, key);
            const int64_t at = (int64_t)t.table[pg] * p.c.page_stride + t.head_off +
                               (int64_t)(key - pg * p.c.page) * p.c.slot_stride;
            const bool see = visible(p, t, key);
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float v = load1<kE4m3>(p.c.v, at + d * 32 + 8 * (r / 4) + 4 * h + (r & 3));
                    st.o[d][r] += see && !(fabsf(v) < INFINITY) ? v : 0.f;
                    __builtin_amdgcn_sched_barrier(0);  // one at a time: registers, not speed
                }
        }
    }
    // Whether this lane's query row sees a position that has a page.
    __device__ static __forceinline__ bool visible(const AttendParams &p, const Task &t, int key) {
        return key <= t.pos && key >= t.lo && key < t.hi &&
               (p.window == 0 || key > t.pos - p.window);
    }

    // One staged tile against the wave's 32 query rows: kSub subtiles of 32
    // keys from subtile `sub` on.
    template <int kSub>
    __device__ static __forceinline__ void compute(Lds &s, int buf, int tile, int sub,
                                                   const AttendParams &p, const Task &t,
                                                   State &st) {
        const int lane = threadIdx.x & (kWave - 1);
        const int h = lane >> 5;
        const int k0 = tile * kTileKeys + sub * 32, k1 = k0 + kSub * 32 - 1;
        const uint32_t *ho = s.marks[buf];
        const uint32_t marks = __builtin_amdgcn_readfirstlane(ho[0] | ho[1] | ho[2] | ho[3]);
        if (k0 > t.pos_max || k0 >= t.hi || k1 < t.lo ||
            (p.window > 0 && k1 <= t.pos_min - p.window))
            return;
        const bool whole = k1 <= t.pos_min && k1 < t.hi && k0 >= t.lo && marks == 0 &&
                           (p.window == 0 || k0 > t.pos_max - p.window);
        const char *kb = s.stage[buf][0] + sub * 32 * D * 2;
        const char *vb = s.stage[buf][1] + sub * 32 * D * 2;
        // scores, transposed: keys down the registers, queries across the lanes
        f32x16 x[kSub];
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[i][r] = 0.f;
        {
            const int row = lane & 31;
            const char *base = kb + row * (D * 2);
            const int f = swizzle<D>(row) ^ h;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
                for (int i = 0; i < kSub; ++i) {
                    const bf16x8 a = *reinterpret_cast<const bf16x8 *>(
                        base + i * 32 * D * 2 + ((f ^ (2 * ks)) << 4));
                    x[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, st.q[ks], x[i], 0, 0, 0);
                }
            }
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const int w = (sub + i) * 2;
                const uint32_t no = (ho[w] & 0xFFFFu) | (ho[w + 1] << 16);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int y = 8 * (r / 4) + 4 * h + (r & 3);
                    const int key = k0 + i * 32 + y;
                    x[i][r] = visible(p, t, key) && !(no >> y & 1) ? x[i][r] : -INFINITY;
                }
            }
        }
        float top = x[0][0];
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, x[i][r]);
        top = half_max(top) * t.c;
        // The maximum only has to keep the exponentials in range: it is raised
        // once a score passes it by 2^8, which few tiles after the first do, and
        // the outputs are rescaled then only.
        if (__any(top > st.m + 8.f)) {
            const float m1 = fmaxf(st.m, top);
            const float keep = m1 == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(st.m - m1);
            st.m = m1;
            st.l *= keep;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) st.o[d][r] *= keep;
        }
        const float m = st.m == -INFINITY ? 0.f : st.m;
        float sum = 0.f;
        bf16x8 w[kSub * 2];
#pragma unroll
        for (int i = 0; i < kSub; ++i) {
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                const float a = __builtin_amdgcn_exp2f(x[i][r] * t.c - m);
                const float b = __builtin_amdgcn_exp2f(x[i][r + 1] * t.c - m);
                sum += a + b;
                const bf16x2 y = __builtin_convertvector((f32x2{a, b}), bf16x2);
                w[2 * i + r / 8][r % 8] = y[0];
                w[2 * i + r / 8][r % 8 + 1] = y[1];
            }
        }
        st.l += sum;
        {
            const int i16 = lane & 15, grp = (lane >> 4) & 1;
            const int f = (2 * grp + ((i16 & 3) >> 1)) ^ (swizzle<D>(i16 >> 2) | h);
            const char *base = vb + (4 * h + (i16 >> 2)) * (D * 2) + (i16 & 1) * 8;
#pragma unroll
            for (int kk = 0; kk < kSub * 2; ++kk) {
#pragma unroll
                for (int d = 0; d < D / 32; ++d) {
                    s16x4 half[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const char *at =
                            base + (16 * kk + 8 * e) * (D * 2) + ((f ^ (4 * d) ^ (2 * e)) << 4);
                        half[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4 *)at);
                    }
                    const s16x8 a = __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7);
                    st.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, a), w[kk], st.o[d], 0, 0, 0);
                }
            }
        }
        if (marks >> 16) add_bad(ho, tile, sub, kSub * 32, p, t, st);
    }

    template <int kSub>
    __device__ static __forceinline__ void run(Lds &s, const AttendParams &p, const Task &t,
                                               int tile, int n, int sub, State &st) {
        Entry e;
        Regs g;
        lookup(p.c, t, tile, e);
        load(p.c, t, tile, e, g);
        if (n > 1) lookup(p.c, t, tile + 1, e);
        store(s, 0, g, partial(p, t, tile));
        for (int i = 0; i < n; ++i) {
            if (i + 1 < n) {
                load(p.c, t, tile + i + 1, e, g);
                if (i + 2 < n) lookup(p.c, t, tile + i + 2, e);
            }
            __syncthreads();
            if (t.active) compute<kSub>(s, i & 1, tile + i, sub, p, t, st);
            // the other buffer's readers passed the barrier above
            if (i + 1 < n) store(s, (i + 1) & 1, g, partial(p, t, tile + i + 1));
        }
        __syncthreads();
    }
};

template <int D, bool kE4m3>
__global__ __launch_bounds__(kTileThreads, kTileWgsPerCu) void attend_tile_kernel(TileParams tp) {
    using T = Tiles<D, kE4m3>;
    __shared__ typename T::Lds s;
    const AttendParams &p = tp.a;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = T::wave_id();
    const int G = p.Hq / p.Hkv, wgs = gridDim.x;

    // tiles before every request
    if (tid == 0) s.before[0] = 0;
    if ((int64_t)p.max_rows * G <= kBlockRows) {
        for (int b = tid; b < p.B; b += kTileThreads) {
            const Request q = load_request(p, b);
            s.before[b + 1] = q.M > 0 ? (uint64_t)block_of(p, q, 0).tiles * p.Hkv : 0;
        }
    } else {
        for (int b = wave; b < p.B; b += kTileWaves) {
            const Request q = load_request(p, b);
            uint64_t n = 0;
            for (int i = lane; i < q.blocks; i += kWave) n += block_of(p, q, i).tiles;
            n = wave_incl_sum_u64(n);
            if (lane == kWave - 1) s.before[b + 1] = n * p.Hkv;
        }
    }
    __syncthreads();
    {
        constexpr int kPer = kGroupRequests / kTileThreads;
        uint64_t x[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid * kPer + i;
            x[i] = b < p.B ? s.before[b + 1] : 0;
            sum += x[i];
        }
        uint64_t in = wave_incl_sum_u64(sum);
        if (lane == kWave - 1) s.part[wave] = in;
        __syncthreads();
        in -= sum;
        for (int i = 0; i < wave; ++i) in += s.part[i];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int b = tid * kPer + i;
            in += x[i];
            if (b < p.B) s.before[b + 1] = in;
        }
    }
    __syncthreads();
    const uint64_t total = s.before[p.B];
    uint64_t per = (uint64_t)udiv64((int64_t)total + wgs - 1, wgs);
    per = per < kMinTiles ? kMinTiles : per;
    // Workgroups go to the 8 XCDs in turn: each XCD takes one run of the tiles, so
    // that units of one head meet in one L2.
    const int used = (int)udiv64((int64_t)(total + per - 1), (int64_t)per);
    const int xcd = blockIdx.x & 7, nth = blockIdx.x >> 3;
    const int share = used / 8 + (xcd < used % 8);
    if (nth >= share) return;
    const int g = xcd * (used / 8) + (xcd < used % 8 ? xcd : used % 8) + nth;
    uint64_t cur = (uint64_t)g * per;
    const uint64_t end = cur + per < total ? cur + per : total;

    // the unit of the first tile
    int b = 0;
    {
        int hi = p.B - 1;
        while (b < hi) {
            const int mid = (b + hi) >> 1;
            if (s.before[mid + 1] <= cur) b = mid + 1;
            else hi = mid;
        }
    }
    Request q = load_request(p, b);
    int head, blk = 0, t0;
    {
        const uint64_t in = cur - s.before[b];
        const uint64_t each = (uint64_t)udiv64((int64_t)(s.before[b + 1] - s.before[b]), p.Hkv);
        head = (int)udiv64((int64_t)in, (int64_t)each);
        uint64_t rest = in - (uint64_t)head * each;
        for (int i0 = 0; q.blocks > 1; i0 += kWave) {
            const int i = i0 + lane;
            const uint64_t n = i < q.blocks ? (uint64_t)block_of(p, q, i).tiles : 0;
            const uint64_t in64 = wave_incl_sum_u64(n);
            const uint64_t all = __shfl(in64, kWave - 1, kWave);
            if (rest < all || i0 + kWave >= q.blocks) {
                const uint64_t after = __ballot(in64 > rest);
                const int first = after ? __ffsll((unsigned long long)after) - 1 : 0;
                blk = i0 + first;
                rest -= __shfl(in64 - n, first, kWave);
                break;
            }
            rest -= all;
        }
        t0 = (int)rest;
    }
    while (cur < end) {
        b = __builtin_amdgcn_readfirstlane(b);
        head = __builtin_amdgcn_readfirstlane(head);
        blk = __builtin_amdgcn_readfirstlane(blk);
        t0 = __builtin_amdgcn_readfirstlane(t0);
        const Block k = block_of(p, q, blk);
        const int left = k.tiles - t0;
        const int n = __builtin_amdgcn_readfirstlane(
            (uint64_t)left < end - cur ? left : (int)(end - cur));
        const int m0 = blk * kBlockRows;
        const int rows = q.M - m0 < kBlockRows ? q.M - m0 : kBlockRows;
        // over 64 rows: a wave per 32 rows, every key; up to 64: two waves per 32
        // rows, each with half of a tile's keys
        const bool wide = rows > 64;
        const int qt = wide ? wave : wave & 1, kg = wide ? 0 : wave >> 1;
        const int mine = qt * 32 + (lane & 31);
        const int m = m0 + mine;
        const bool valid = mine < rows;
        const int j = m / G;
        const int64_t row = q.start + j;
        const int hq = head * G + (m - j * G);

        typename T::Task t;
        t.table = p.c.table + (int64_t)b * p.c.table_width;
        t.head_off = (int64_t)head * p.c.head_stride;
        t.lo = k.lo;
        t.hi = k.hi;
        t.ctx = q.ctx;
        t.pos = q.ctx + j;
        t.first = q.ctx + m0 / G;
        t.final = q.ctx + (m0 + rows - 1) / G;
        t.pos_min = q.ctx + (m0 + qt * 32) / G;
        const int m_last = (qt * 32 + 31 < rows - 1 ? qt * 32 + 31 : rows - 1) + m0;
        t.pos_max = q.ctx + m_last / G;
        t.active = qt * 32 < rows;
        // a negative scale turns the queries' signs, none at all their values to 0
        const float scale = p.scale * p.c.k_scale;
        t.c = (scale == 0.f ? 1.f : fabsf(scale)) * kLog2e;
        const uint32_t keep = scale == 0.f ? 0u : 0xFFFFFFFFu;
        const uint32_t flip = scale < 0.f ? 0x80008000u : 0u;

        typename T::State st;
        st.m = -INFINITY;
        st.l = 0.f;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) st.o[d][r] = 0.f;
        {
            const uint16_t *src = p.q + row * p.q_row + hq * p.q_head + (lane >> 5) * 8;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                u32x4 x = {0u, 0u, 0u, 0u};
                if (valid) x = *reinterpret_cast<const u32x4 *>(src + ks * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = (x[i] & keep) ^ flip;
                st.q[ks] = __builtin_bit_cast(bf16x8, x);
            }
        }
        if (wide) T::template run<2>(s, p, t, k.tile + t0, n, 0, st);
        else T::template run<1>(s, p, t, k.tile + t0, n, kg, st);
        st.l = half_sum(st.l);

        if (!wide) {  // the two halves of the keys meet
            float *mem = s.join[qt];
            if (kg == 1 && t.active) {
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) mem[(d * 16 + r) * kWave + lane] = st.o[d][r];
                mem[(D / 2) * kWave + lane] = st.m;
                mem[(D / 2 + 1) * kWave + lane] = st.l;
            }
            __syncthreads();
            if (kg == 0 && t.active) {
                const float om = mem[(D / 2) * kWave + lane], ol = mem[(D / 2 + 1) * kWave + lane];
                const float top = fmaxf(st.m, om);
                const float a = st.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.m - top);
                const float c = om == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(om - top);
                st.m = top;
                st.l = st.l * a + ol * c;
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        st.o[d][r] = st.o[d][r] * a + mem[(d * 16 + r) * kWave + lane] * c;
            }
            __syncthreads();
        }
        const bool owner = kg == 0 && t.active && valid;
        if (n == k.tiles) {
            if (owner) {
                const float norm = st.l > 0.f ? p.c.v_scale / st.l : 0.f;
                uint16_t *o = p.out + (row * p.Hq + hq) * D + (lane >> 5) * 4;
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        const uint64_t y =
                            (uint64_t)pack_bf16(st.o[d][r] * norm, st.o[d][r + 1] * norm) |
                            ((uint64_t)pack_bf16(st.o[d][r + 2] * norm, st.o[d][r + 3] * norm)
                             << 32);
                        *reinterpret_cast<uint64_t *>(o + d * 32 + 2 * r) = y;
                    }
            }
        } else {
            const uint64_t unit = cur - t0;
            const int g0 = (int)udiv64((int64_t)unit, (int64_t)per);
            const int g1 = (int)udiv64((int64_t)(unit + k.tiles - 1), (int64_t)per);
            const int64_t slot = slot_floats(tp.slot_rows, D);
            auto slot_of = [&](int w) { return tp.slots + slot * (2 * (int64_t)w + (w == g0)); };
            if (owner) {
                float *to = slot_of(g);
                if (lane < 32) store_coherent(to + 2 * mine, st.m, st.l);
                to += 2 * tp.slot_rows + (int64_t)mine * D + (lane >> 5) * 4;
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        store_coherent(to + d * 32 + 2 * r, st.o[d][r], st.o[d][r + 1]);
                        store_coherent(to + d * 32 + 2 * r + 2, st.o[d][r + 2], st.o[d][r + 3]);
                    }
            }
            __builtin_amdgcn_s_waitcnt(0);  // the partial results are at the coherence point
            __syncthreads();
            if (tid == 0) {
                const unsigned old = __hip_atomic_fetch_add(tp.arrivals + g0, (unsigned)n,
                                                            __ATOMIC_RELAXED,
                                                            __HIP_MEMORY_SCOPE_AGENT);
                s.last = old + (unsigned)n == (unsigned)k.tiles;
                if (s.last)  // zero again for the next call
                    __hip_atomic_store(tp.arrivals + g0, 0u, __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
            }
            __syncthreads();
            if (s.last) {
                for (int i = tid; i < rows * (D / 2); i += kTileThreads) {
                    const int x = i / (D / 2), d = 2 * (i - x * (D / 2));
                    float top = -INFINITY;
                    for (int w = g0; w <= g1; ++w)
                        top = fmaxf(top, load_coherent(slot_of(w) + 2 * x)[0]);
                    float l = 0.f, a = 0.f, c = 0.f;
                    for (int w = g0; w <= g1; ++w) {
                        const float *from = slot_of(w);
                        const f32x2 ml = load_coherent(from + 2 * x);
                        const f32x2 v =
                            load_coherent(from + 2 * tp.slot_rows + (int64_t)x * D + d);
                        const float f =
                            ml[0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[0] - top);
                        l += f * ml[1];
                        a += f * v[0];
                        c += f * v[1];
                    }
                    const float norm = l > 0.f ? p.c.v_scale / l : 0.f;
                    const int jj = (m0 + x) / G, hh = head * G + (m0 + x - jj * G);
                    *reinterpret_cast<uint32_t *>(
                        p.out + ((int64_t)(q.start + jj) * p.Hq + hh) * D + d) =
                        pack_bf16(a * norm, c * norm);
                }
            }
        }
        // the next unit
        cur += n;
        t0 = 0;
        if (cur < end) {
            if (++blk == q.blocks) {
                blk = 0;
                if (++head == p.Hkv) {
                    head = 0;
                    do q = load_request(p, ++b);
                    while (q.blocks == 0);
                }
            }
        }
    }
}

static int tile_wgs() { return kTileWgsPerCu * device_cu_count(); }
static int tile_slot_rows(int max_rows, int Hq, int Hkv) {
    const int64_t m = (int64_t)max_rows * (Hq / Hkv);
    return m >= kBlockRows ? kBlockRows : (int)((m + 31) / 32 * 32);
}
static size_t tile_arrival_bytes() { return ((size_t)tile_wgs() * 4 + 255) & ~(size_t)255; }

size_t attention_ws_bytes(int B, int max_rows, int Hq, int Hkv, int D) {
    (void)B;
    if (D != 64 && D != 128) return 256;
    const size_t n = tile_arrival_bytes() +
                     (size_t)2 * tile_wgs() *
                         (size_t)slot_floats(tile_slot_rows(max_rows, Hq, Hkv), D) * 4;
    return (n + 255) & ~(size_t)255;
}

template <int D, bool kE4m3>
static hipError_t launch_tiles(const AttendParams &p, void *ws, hipStream_t s) {
    TileParams tp;
    tp.a = p;
    tp.arrivals = static_cast<unsigned *>(ws);
    tp.slots = reinterpret_cast<float *>(static_cast<char *>(ws) + tile_arrival_bytes());
    tp.slot_rows = tile_slot_rows(p.max_rows, p.Hq, p.Hkv);
    for (int b = 0; b < p.B; b += kGroupRequests) {
        tp.a.B = p.B - b < kGroupRequests ? p.B - b : kGroupRequests;
        tp.a.cu = p.cu + b;
        tp.a.ctx = p.ctx + b;
        tp.a.c.table = p.c.table + (int64_t)b * p.c.table_width;
        hipLaunchKernelGGL((attend_tile_kernel<D, kE4m3>), dim3(tile_wgs()), dim3(kTileThreads), 0,
                           s, tp);
    }
    return hipGetLastError();
}

hipError_t launch_attention(const AttendParams &p, bool e4m3, void *ws, hipStream_t s) {
    if (p.D == 128)
        return e4m3 ? launch_tiles<128, true>(p, ws, s) : launch_tiles<128, false>(p, ws, s);
    if (p.D == 64)
        return e4m3 ? launch_tiles<64, true>(p, ws, s) : launch_tiles<64, false>(p, ws, s);
    const dim3 grid((unsigned)p.rows, (unsigned)p.Hq);
    if (e4m3) hipLaunchKernelGGL((attend_row_kernel<true>), grid, dim3(kRowThreads), 0, s, p);
    else hipLaunchKernelGGL((attend_row_kernel<false>), grid, dim3(kRowThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace dspark
