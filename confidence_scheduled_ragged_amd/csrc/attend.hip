// attend.hip - attention of the packed verify rows over each request's pages of
// the key-value cache.
//
// Row j of request b stands at position p = ctx[b] + j and sees the positions
// max(0, p - window + 1) .. p (from 0 without a window) whose page the table
// names:
//   O = sum_t exp(x_t - m) V_t / sum_t exp(x_t - m),  x_t = scale (q . K_t),
// with m the largest x_t. A running maximum and sum carry the softmax over the
// keys in one pass; a row that sees nothing gives zeros.
//
// Compiled twice: as is, for rows in a chain, and with DSPARK_TREE=1 for the nodes of
// drafted trees and for windows with first positions that stay visible (the rows that
// TreeView describes). One kernel for both would cost the chains registers.
#include <type_traits>

#include "forward.hpp"

#ifndef DSPARK_TREE
#define DSPARK_TREE 0
#endif

namespace dspark {
#if DSPARK_TREE
namespace trees {
#else
namespace chains {
#endif

constexpr bool kTree = DSPARK_TREE;

constexpr int kMaxHeadDim = 256;
constexpr int kRowThreads = 64;

// Contexts are taken as at most this many positions, so that those of the call's
// rows (2^24 at most) and of a tile past them fit in 32 bits.
constexpr int kMaxContext = 0x7FFFFFFF - (1 << 25) + 1;
static_assert(DSPARK_MAX_ROWS <= 1 << 24, "positions of the rows");
__device__ __forceinline__ int context_of(int ctx) {
    return ctx < 0 ? 0 : (ctx > kMaxContext ? kMaxContext : ctx);
}

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

// Any head size and alignment: one wave per (packed row, query head), 64 keys at a
// time, a lane per key for the scores and a lane per output element for the
// weighted values. Bound by its latency: 32 requests of mixed traffic at D = 96 took
// 2127 us here and take 66 us in the tiles below, so only heads over 128 and pools
// that 16-byte loads do not fit come here. Keys and values are read again for every row
// and query head: one tree of 60 nodes on 4000 positions with 8 + 2 heads of 256 takes
// 4.4 ms, 32 trees of 12 to 32 nodes 3.7 ms; 45 us the latter with 16 + 4 heads of 128,
// as many bytes, in the tiles.
template <bool kE4m3>
__global__ __launch_bounds__(kRowThreads) void attend_row_kernel(AttendParams p, TreeView v) {
    __shared__ float q_s[kMaxHeadDim];
    __shared__ float p_s[kWave];
    __shared__ int64_t at_s[kWave];
    const int lane = threadIdx.x;
    const int r = blockIdx.x, h = blockIdx.y;
    const int b = wave_request_of(p.cu, p.B, r);
    if (b >= p.B) return;
    const int first = p.cu[b], j = r - first;
    if (j < 0 || j >= p.max_rows) return;
    const int kvh = h / (p.Hq / p.Hkv);
    const bool masked = kTree && v.masks;
    // positions past the table's width have no page
    const int64_t width = (int64_t)p.c.table_width * p.c.page;
    const int64_t ctx = context_of(p.ctx[b]);
    const int64_t pos = ctx + (masked ? depth_of(v.depths, r, j) : j);
    int64_t last = pos + 1;  // and the first position in the window
    int64_t begin = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
    const uint32_t *mask = nullptr;
    if (masked) {
        const int rows = p.cu[b + 1] < p.rows ? p.cu[b + 1] - first : p.rows - first;
        last = ctx + (rows < p.max_rows ? rows : p.max_rows);
        begin = begin < ctx ? begin : ctx;
        mask = v.masks + (int64_t)r * v.words;
    }
    const int64_t end = last < width ? last : width;
    const int64_t sinks = !kTree ? 0 : (v.sinks < begin ? v.sinks : begin);
    const int64_t sinks_end = sinks < width ? sinks : width;
    const int32_t *row = p.c.table + (int64_t)b * p.c.table_width;
    const uint16_t *q = p.q + r * p.q_row + h * p.q_head;
    for (int d = lane; d < p.D; d += kWave) q_s[d] = bf16_f32(q[d]) * p.scale * p.c.k_scale;
    __syncthreads();
    float m = -INFINITY, total = 0.f;
    float acc[kMaxHeadDim / kWave] = {};
    auto keys = [&](int64_t t0, int64_t t1) {
        const int64_t t = t0 + lane;
        bool see = t < t1;
        if (masked && see && t >= ctx) see = mask[(t - ctx) >> 5] >> ((t - ctx) & 31) & 1;
        const int64_t at = see ? slot_offset(p.c, row, (int)t, kvh) : -1;
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
        // fmaxf drops NaN: keys may be there that leave no maximum
        if (!__any(at >= 0)) return;
        const float m1 = fmaxf(m, top);
        const float base = m1 == -INFINITY ? 0.f : m1;
        const float keep = expf(m - base);  // 0 before the first maximum
        const float w = at >= 0 ? expf(x - base) : 0.f;
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
    };
    for (int64_t t = 0; t < sinks_end; t += kWave) keys(t, sinks_end);
    for (int64_t t = begin; t < end; t += kWave) keys(t, end);
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
// head, a request's n rows are M = n*G query rows, taken in blocks of up to 128 or
// 256 against tiles of 64 to 256 positions (32 KiB of keys and values). A (head,
// block) is a unit; the tiles of all units, laid end to end with a few places
// ahead of each unit's for what it costs beside them, are divided evenly between
// the resident workgroups, so any mix of long and short requests fills the chip, a
// single long context included, and no launch shape depends on the lengths. A unit
// that ends up in several workgroups leaves partial results (maximum, sum, weighted
// values) in the workspace; of a chain, the last workgroup to arrive joins them in
// tile order, of trees, which have more rows, join_kernel does.
//
// Tiles are loaded from the pages straight into LDS, ahead of the tile at work and
// whatever unit they belong to. Through registers, the loads alone took 326 of the
// 409 us of a mixed batch (256 requests, 1.33 GB of keys and values) and 405 of the
// 831 us of a prompt's chunk (2048 rows on 14000 positions). Calls of up to 128 query
// rows a head (decoding, verify windows) have two workgroups of four waves a CU, a
// tile at work and one on its way in each. The mixed batch takes 302 us, 4.4 TB/s
// (its loads alone 242 us, 5.5 TB/s: the products, and units that begin and end, are
// not all behind them); four contexts of 40000 to 120000 in 8 bits 147 us, 4.4 TB/s
// (loads alone 137 us, 4.7 TB/s, by what two tiles keep on their way); one token at
// 4000, a chain of some ten round trips to memory, 21 us (14). Calls with more
// (prompts) are bound by the matrix and vector instructions of the softmax, which
// two waves of a SIMD overlap poorly: one workgroup of eight waves a CU, four tiles in
// LDS, so that keys are read from L2 once for 256 rows. The chunk takes 602 us, 837
// TFLOP/s (loads alone 199 us), four prompts of 1882 to 2902 tokens 312 us, 671
// TFLOP/s (99 us); in 8 bits these prompts take 347 us, since that kernel spills 25
// registers, whose reloads wait behind the loads into LDS. Figures of one card;
// others took 1 to 5 % more or less.
//
// Trees and sinks (DSPARK_TREE=1): 128 trees of 12 to 32 nodes, G = 4, take 178 us, 15
// of them in the join. Where each workgroup has one whole unit, of 64 trees of 12 (24)
// nodes in windows of 256 to 2048, a tile takes 3.3 (3.9) us with all of them loading,
// 5.1 (4.3) TB/s; a second unit takes 5 to 9 us beside its tiles. Four trees of 64 nodes
// on 41 to 113 thousand positions in 8 bits take 449 us, 834 TFLOP/s. One tree of 60
// nodes on 4000 takes 31 us, a chain of waits: the tiles' kernel 16 us where units have
// one tile, 2.1 for each further one up to the five that a workgroup takes at least, 28
// on 4000, then 4 for the join. Trees of more than 64 nodes read their masks' words from
// memory, behind the tiles on their way: 64 of 100 to 256 nodes on 128 to 4096 positions
// take 529 us, 3.0 times what their operations need; 64 of 32 to 64 nodes take 172, 2.3
// times what their bytes need.
//
// Scores are computed transposed, S^T = K Q^T: a lane then holds 16 of a query's 32
// scores of one MFMA (the other 16 sit in lane ^ 32), so the softmax needs one
// exchange between the halves, and the weights leave the exponential in the
// very places where the next product, O^T = V^T P^T, wants them. V^T comes
// from row-major V in LDS through the transposing LDS reads. 8-bit tiles stay as
// they are in LDS and are widened, exactly, on their way to the matrix product.
//
// Weights are rounded to bf16 before their product with V (half a step 2^-8 of
// each weight, averaged over the keys); sums, maxima and outputs stay in fp32.

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr int kNarrowRows = 128, kWideRows = 256;  // query rows of a block
constexpr int kSlotBytes = 32768;                  // of a tile in LDS: keys, then values
constexpr int kHalfSlot = kSlotBytes / 2;
constexpr int kGroupRequests = 512;  // of one launch; larger batches take several
constexpr int kMinTiles = 1;  // per workgroup; one token at 4000 takes 21.5 us with 1, 22.5 with 2
constexpr int kZeroBytes = 256;       // of the workspace that stay zero
// kUnitTiles (below) of trees, whose cuts cost less: at 1, 2, 3, 4 and 5 128 trees took
// 199, 186, 174, 173 and 170 us, four prompts in a window 269, 262, 250, 254 and 257 us.
constexpr int kTreeUnitTiles = 4;
constexpr float kLog2e = 1.44269504088896340736f;

struct TileParams {
    AttendParams a;
    const char *zeros;   // kZeroBytes
    unsigned *arrivals;  // [wgs], zero between calls
    float *slots;        // [2 * wgs] partial results of slot_rows rows
    int slot_rows;
    // 16 slots in a row share a page, and a page and 16 slots are below 2^32 bytes
    bool together;
    uint32_t page_bytes, slot_bytes;
#if DSPARK_TREE
    TreeView v;
    struct Split *splits;  // of every unit, or of every workgroup: [wgs] at most
    int blocks;            // the most of a request, where there is one for every unit; or 0
#endif
};

// A unit that is cut after its first workgroup's tiles: its parts are in the slots of
// workgroups first .. first + parts - 1. No parts where none is. Few units have one
// each, of many each workgroup has one, for the unit that it is the first to cut.
struct Split {
    int parts, first, rows, head, start, m0;
    int pad[2];
};

// The call's parameters, read again from the kernel's arguments: for what runs once
// a unit or less. Kept from the start, they would push the scalars of every tile
// out of the registers.
__device__ __forceinline__ TileParams params_again() {
    struct Words {
        uint32_t w[sizeof(TileParams) / 4];
    } words;
    uint64_t at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(at));
#pragma unroll
    for (unsigned i = 0; i < sizeof(TileParams) / 4; ++i)
        words.w[i] = ((const __attribute__((address_space(4))) uint32_t *)at)[i];
    return __builtin_bit_cast(TileParams, words);
}

// Floats of one partial result: (maximum, sum) and D values of each row.
__host__ __device__ inline int64_t slot_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

// The lengths and the table are read by scalar loads, apart from the loads into
// LDS, which return in order.
typedef const __attribute__((address_space(4))) int32_t *ScalarInts;
__device__ __forceinline__ int scalar_load(const int32_t *p, int64_t i) {
    return ((ScalarInts)(uintptr_t)p)[i];
}

struct Request {
    int start, ctx, M, blocks;
};
__device__ __forceinline__ Request request_of(const AttendParams &p, int log_rows, int s, int e,
                                              int c) {
    Request q;
    s = s < 0 ? 0 : (s > p.rows ? p.rows : s);
    e = e < s ? s : (e > p.rows ? p.rows : e);
    const int n = e - s < p.max_rows ? e - s : p.max_rows;
    q.start = s;
    q.ctx = context_of(c);
    q.M = n * (p.Hq / p.Hkv);
    q.blocks = (q.M + (1 << log_rows) - 1) >> log_rows;
    return q;
}
__device__ __forceinline__ Request load_request(const AttendParams &p, int log_rows, int b) {
    return request_of(p, log_rows, p.cu[b], p.cu[b + 1], p.ctx[b]);
}
__device__ __forceinline__ Request scalar_request(const AttendParams &p, int log_rows, int b) {
    return request_of(p, log_rows, scalar_load(p.cu, b), scalar_load(p.cu, b + 1),
                      scalar_load(p.ctx, b));
}
// Positions [lo, hi) that block i of a request needs, its first and last row's
// positions, and its tiles (one at least: a block that sees nothing still writes
// its zeros). Rows with masks may see any row of their request, so that only the
// context is common to all; their positions are at most the last row's. `sink` tiles
// from the first on stay visible below the window's.
struct Block {
    int lo, hi, first, final, tile, tiles;
#if DSPARK_TREE
    int sink;
#endif
    // the i-th tile
    __device__ __forceinline__ int at(int i) const {
#if DSPARK_TREE
        return i < sink ? i : tile + i - sink;
#else
        return tile + i;
#endif
    }
    __device__ __forceinline__ int after(int t) const {  // the tile after tile t
#if DSPARK_TREE
        return t + 1 == sink && t + 1 < tile ? tile : t + 1;
#else
        return t + 1;
#endif
    }
};
template <int kKeys>
__device__ __forceinline__ Block block_of(const TileParams &tp, int log_rows, const Request &q,
                                          int i) {
    const AttendParams &p = tp.a;
    const int G = p.Hq / p.Hkv;
    const int m0 = i << log_rows;
    const int m1 = (q.M < m0 + (1 << log_rows) ? q.M : m0 + (1 << log_rows)) - 1;
    const int64_t width = (int64_t)p.c.table_width * p.c.page;
    Block k;
    k.first = q.ctx + m0 / G;
    k.final = q.ctx + m1 / G;
#if DSPARK_TREE
    if (tp.v.masks) {
        k.first = q.ctx;
        k.final = q.ctx + q.M / G - 1;
    }
#endif
    k.lo = 0;
    if (p.window > 0 && k.first + 1 > p.window) k.lo = k.first + 1 - p.window;
    const int end = k.final + 1;
    k.hi = end < width ? end : (int)width;
    k.tile = k.lo / kKeys;
    const int last = (int)(((int64_t)k.hi + kKeys - 1) / kKeys);
    k.tiles = last > k.tile ? last - k.tile : 0;
#if DSPARK_TREE
    if (tp.v.masks) k.first = q.ctx - 1;
    const int sinks = tp.v.sinks < k.hi ? tp.v.sinks : k.hi;
    const int sink = (sinks + kKeys - 1) / kKeys;
    k.sink = sink < k.tile ? sink : k.tile;
    k.tiles += k.sink;
#endif
    if (k.tiles == 0) k.tiles = 1;
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

// Waits until at most kLoads of this wave's vector loads are on their way and its
// LDS accesses are done.
template <int kLoads>
__device__ __forceinline__ void wait_loads() {
    __builtin_amdgcn_s_waitcnt((kLoads & 15) | (7 << 4) | ((kLoads >> 4) << 14));
}

// Chunk (16 bytes) c of row r of a staged tile sits at chunk c ^ swizzle(r), so
// that the score operand (one chunk of 32 rows) and the transposed reads (8 or
// 16 rows of two to four chunks) each meet few equal banks.
template <int D, bool kE4m3>
__device__ __forceinline__ int swizzle(int r) {
    if (!kE4m3 && D == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
    if (!kE4m3) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    if (D == 128) return ((r >> 2) & 1) | (r & 2) | (((r >> 3) & 1) << 2);
    return (r >> 2) & 3;
}

// D is the head size that the tiles are made for; with kPadded the heads are
// shorter, and the elements between come from the zeros.
template <int D, bool kE4m3, bool kWide, bool kPadded>
struct Tiles {
    static constexpr int kWaves = kWide ? 8 : 4;
    static constexpr int kThreads = kWaves * kWave;
    static constexpr int kSlots = kWide ? 4 : 2;         // tiles in LDS
    static constexpr int kLogRows = kWide ? 8 : 7;  // query rows of a block
    static_assert((kWide ? kWideRows : kNarrowRows) == 1 << kLogRows, "blocks");
    // What a unit costs beside its tiles (its queries, its first tile, joining and
    // storing its rows), in tiles: a unit has this many places, then its tiles. At 0,
    // 1, 2, 3 and 5 the mixed batch took 377, 346, 315, 307 and 313 us, four prompts
    // 378, 367, 350, 333 and 318 us.
    static constexpr int kUnitTiles = kWide ? 5 : 3;
    static constexpr int kItem = kE4m3 ? 1 : 2;
    static constexpr int kRow = D * kItem;               // bytes
    static constexpr int kChunks = kRow / 16;            // of a row
    static constexpr int kKeys = kHalfSlot / kRow;       // positions of a tile
    static constexpr int kLoadRows = kWave / kChunks;    // rows of one load (4, 8 or 16)
    static constexpr int kStagers = kWaves / 2;          // waves that stage keys, and values
    static constexpr int kWaveRows = kKeys / kStagers;   // rows that each of them stages
    static constexpr int kWaveLoads = kHalfSlot / kStagers / 1024;  // of 1 KiB
    static constexpr int kEntries = kWaveRows / 16;      // 16 rows each
    static constexpr int kRowWords = (kWaveRows + 63) / 64;  // of a bit for each of them
    static_assert(64 % kLoadRows == 0 && (kRowWords == 1 || kWaveRows % 64 == 0),
                  "the rows of a load share a word");

    struct Lds {
        uint64_t before[kGroupRequests + 1];
        uint64_t part[kWaves];
        float join[16 * (kWaves / 2) * kWave];
        f32x2 ml[kWaves / 2 * kWave];
        // rows whose values were not all finite, per staging wave
        uint64_t bad[kSlots][kStagers * kRowWords];
#if DSPARK_TREE
        uint64_t bits[kThreads];  // of each lane's row, where 64 are enough
#endif
        int last;
    };

    // The tiles in LDS are variables of their own, not one array: the compiler
    // then knows which loads into LDS a read of keys has to wait for, where the slot
    // is chosen by a branch.
    struct Slots {
        char *at0, *at1, *at2, *at3;
        template <typename F>
        __device__ __forceinline__ void pick(int n, F f) const {
            if (kSlots == 2 || n < 2) {
                if (n == 0) f(at0);
                else f(at1);
            } else if (n == 2) {
                f(at2);
            } else {
                f(at3);
            }
        }
        __device__ static __forceinline__ uint32_t address(const char *p) {
            uint32_t a = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)p;
            asm("" : "+s"(a));  // or the choice becomes a table, which LDS addresses cannot fill
            return a;
        }
        __device__ __forceinline__ uint32_t address(int n) const {
            return kSlots == 2 || n < 2 ? (n == 0 ? address(at0) : address(at1))
                                        : (n == 2 ? address(at2) : address(at3));
        }
    };

    // A unit, and the tiles of it from `tile` on that are this workgroup's.
    struct Unit {
        int b, head, blk;
        Request q;
        Block k;
        int tile, left;  // next tile; tiles left in the unit
    };
    // The wave's part of a unit.
    struct Task {
        const int32_t *table;
        int64_t head_off;      // of the key-value head in the pools
        int lo, hi, first, final;
        int pos;               // of this lane's query row
        int pos_min, pos_max;  // over the wave's query rows
        bool active, hole;     // hole: some position may have no page
        float c;               // scores to powers of two
#if DSPARK_TREE
        int border;            // positions from here on are seen by the row's bits
        int sinks;
        const uint32_t *mask;  // of the row, where it has more than 64 bits
#endif
    };
    struct State {
        bf16x8 q[D / 16];
        f32x16 o[D / 32];
        float m, l;
    };

    __device__ static __forceinline__ int wave_id() {
        return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    }
    __device__ static __forceinline__ bool named(const PagedCache &c, int at) {
        return at >= 0 && at < c.pages;
    }

    // ------------------------------------------------------------- staging
    struct Stager {
        const char *base;          // the unit's head in the pool of keys or values
        const int32_t *table;      // the unit's pages
        int row0;                  // of the wave's rows in a tile
        uint32_t off[kWaveLoads];  // this lane's bytes from the first of 16 rows
        // pages of the wave's rows, 16 each, in tiles batch0 + lane: one load for 64
        // tiles, since a wait for it waits for the tiles on their way too
        int batch[kEntries];
        int batch0;
    };
    // The chunk of its row that a lane fetches in load j.
    __device__ static __forceinline__ int chunk_of(int lane, int j) {
        return (lane % kChunks) ^ swizzle<D, kE4m3>(j * kLoadRows + lane / kChunks);
    }
    __device__ static __forceinline__ void stager(const TileParams &tp, Stager &g) {
        const PagedCache &c = tp.a.c;
        const int lane = threadIdx.x & (kWave - 1), w = wave_id();
        g.row0 = w % kStagers * kWaveRows;
#pragma unroll
        for (int j = 0; j < kWaveLoads; ++j) {
            const int r = j * kLoadRows + lane / kChunks;
            g.off[j] = (uint32_t)(r % 16) * tp.slot_bytes + (chunk_of(lane, j) << 4);
        }
    }
    __device__ static __forceinline__ void enter(const TileParams &tp, Stager &g, const Unit &u) {
        const PagedCache c = params_again().a.c;
        g.base = static_cast<const char *>(wave_id() < kStagers ? c.k : c.v) +
                 (int64_t)u.head * c.head_stride * kItem;
        g.table = c.table + (int64_t)u.b * c.table_width;
    }
    __device__ static __forceinline__ void look_up(const TileParams &tp, Stager &g, int tile) {
        const PagedCache c = params_again().a.c;
        const int lane = threadIdx.x & (kWave - 1);
        g.batch0 = tile;
        if (!tp.together) return;
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int64_t pos = (int64_t)(tile + lane) * kKeys + g.row0 + 16 * e;
            const int pg = pos > 0x7FFFFFFF ? c.table_width : page_of(c, (int)pos);
            g.batch[e] = pg < c.table_width ? g.table[pg] : -1;
        }
    }
    __device__ static __forceinline__ void dma(const char *from, char *to) {
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void *)from,
            (__attribute__((address_space(3))) void *)to, 16, 0, 0);
    }
    // The wave's loads of one tile into a slot. Rows without a page come from the
    // zeros. Rows of a page that lie outside [lo, hi) are loaded as they are: they
    // are masked like rows that a query does not see.
    __device__ static __forceinline__ void issue(const TileParams &tp, const Stager &g, int tile,
                                                 const Slots &slots, int number, int lane) {
        const PagedCache &c = tp.a.c;
        const int w = wave_id();
        const char *from[kWaveLoads];
        if (tp.together) {
#pragma unroll
            for (int e = 0; e < kEntries; ++e) {
                const int at = __builtin_amdgcn_readlane(g.batch[e], tile - g.batch0);
                const bool ok = (unsigned)at < (unsigned)c.pages;
                const int pos = tile * kKeys + g.row0 + 16 * e;
                const uint32_t slot = (uint32_t)(pos - page_of(c, pos) * c.page);
                const char *base = ok ? g.base + (uint64_t)(uint32_t)at * tp.page_bytes +
                                            slot * tp.slot_bytes
                                      : tp.zeros;
#pragma unroll
                for (int j = e * kWaveLoads / kEntries; j < (e + 1) * kWaveLoads / kEntries; ++j)
                    from[j] = base + (ok ? g.off[j] : (uint32_t)(lane & 15) * 16);
            }
            if constexpr (kPadded) {
#pragma unroll
                for (int j = 0; j < kWaveLoads; ++j)
                    if (chunk_of(lane, j) * 16 >= tp.a.D * kItem)
                        from[j] = tp.zeros + (lane & 15) * 16;
            }
        } else {
            const TileParams cold = params_again();
#pragma unroll
            for (int j = 0; j < kWaveLoads; ++j) {
                const int r = j * kLoadRows + lane / kChunks;
                const int64_t at = slot_offset(cold.a.c, g.table, tile * kKeys + g.row0 + r, 0);
                from[j] = at < 0 || (kPadded && chunk_of(lane, j) * 16 >= cold.a.D * kItem)
                              ? cold.zeros
                              : g.base + at * kItem + (chunk_of(lane, j) << 4);
            }
        }
        slots.pick(number, [&](char *slot) {
#pragma unroll
            for (int j = 0; j < kWaveLoads; ++j)
                dma(from[j], slot + (w * kWaveLoads + j) * 1024);
        });
    }

    // Whether some row of the block does not see some key of the tile that another
    // one sees, or the tile holds rows that none sees. There a weight of zero must
    // keep out whatever the value is, which zero times an infinity or NaN would
    // not: values that are not finite are set to 0 in LDS, and add_bad adds them to
    // the rows that see them.
    __device__ static __forceinline__ bool partial(const AttendParams &p, const Task &t, int tile) {
        const int k0 = tile * kKeys;
#if DSPARK_TREE
        if (k0 + kKeys <= t.sinks) return k0 + kKeys - 1 > t.first;
#endif
        return k0 + kKeys - 1 > t.first || (p.window > 0 && k0 <= t.final - p.window);
    }
    __device__ static __forceinline__ bool bad_word(uint32_t x) {
        if (kE4m3) {  // a byte of 0x7F without its sign
            const uint32_t y = (x & 0x7F7F7F7Fu) ^ 0x7F7F7F7Fu;
            return ((y - 0x01010101u) & ~y & 0x80808080u) != 0;
        }
        return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
    }
    __device__ static __forceinline__ uint32_t good_part(uint32_t x) {
        if (kE4m3) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((x >> (8 * i) & 0x7Fu) == 0x7Fu) x &= ~(0xFFu << (8 * i));
            return x;
        }
        if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
        if ((x & 0x7F800000u) == 0x7F800000u) x &= 0xFFFFu;
        return x;
    }
    // By each wave that stages values, on its own rows, once they have arrived.
    __device__ static __forceinline__ void scrub(Lds &s, const Slots &slots, int n, int lane) {
        const int w = wave_id();
        if (w < kStagers) return;
        uint64_t rows[kRowWords] = {};
        typedef __attribute__((address_space(3))) u32x4 *Words;
        const uint32_t slot = slots.address(n);
#pragma unroll 1
        for (int j = 0; j < kWaveLoads; ++j) {
            const Words at = (Words)(uintptr_t)(slot + (w * kWaveLoads + j) * 1024 + lane * 16);
            u32x4 x = *at;
            const bool bad = bad_word(x[0]) || bad_word(x[1]) || bad_word(x[2]) || bad_word(x[3]);
            const uint64_t m = __ballot(bad);
            if (m == 0) continue;
            if (bad) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = good_part(x[i]);
                *at = x;
            }
            uint64_t here = 0;
            for (int r = 0; r < kLoadRows; ++r)
                if (m >> (r * kChunks) & ((1ull << kChunks) - 1))
                    here |= 1ull << (j * kLoadRows % 64 + r);
#pragma unroll
            for (int i = 0; i < kRowWords; ++i)
                if (j * kLoadRows / 64 == i) rows[i] |= here;
        }
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kRowWords; ++i) s.bad[n][(w - kStagers) * kRowWords + i] = rows[i];
        }
        wait_loads<63>();  // LDS accesses only
    }
    // The values that scrub left out of 32 keys, from the cache again: to the
    // rows that see them. Their weights do not matter: the sum is not finite with
    // any.
    __device__ static __forceinline__ void add_bad(const uint64_t *bad, int tile, int sub,
                                                   const AttendParams &p, const Task &t,
                                                   State &st, const Lds &s, int lane) {
        const int h = lane >> 5;
        const AttendParams cold = params_again().a;
#if DSPARK_TREE
        const uint32_t bits = seen(p, s, t, tile * kKeys + sub * 32);
#endif
#pragma unroll 1
        for (int y = sub * 32; y < sub * 32 + 32; ++y) {
            if (!(bad[y / kWaveRows * kRowWords + y % kWaveRows / 64] >> (y % kWaveRows % 64) & 1))
                continue;
            const int key = tile * kKeys + y;
            const int64_t at = slot_offset(cold.c, t.table, key, 0);
            if (at < 0) continue;
#if DSPARK_TREE
            const bool see = bits >> (y & 31) & 1;
#else
            const bool see = visible(p, t, key);
#endif
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int e = d * 32 + 8 * (r / 4) + 4 * h + (r & 3);
                    if (kPadded && e >= cold.D) continue;
                    const float v = load1<kE4m3>(cold.c.v, at + t.head_off + e);
                    st.o[d][r] += see && !(fabsf(v) < INFINITY) ? v : 0.f;
                    __builtin_amdgcn_sched_barrier(0);  // one at a time: registers, not speed
                }
        }
    }

    // ------------------------------------------------------------- compute
#if DSPARK_TREE
    // Bits below n of 32.
    __device__ static __forceinline__ uint32_t below(int n) {
        return n >= 32 ? 0xFFFFFFFFu : (1u << (n < 0 ? 0 : n)) - 1u;
    }
    // The positions of 32 from k0 on that this lane's query row sees, if they have pages,
    // as bits. Up to 64 bits of the row's mask are kept in LDS: a load from memory, which
    // more of them take, waits for the tiles on their way.
    __device__ static __forceinline__ uint32_t seen(const AttendParams &p, const Lds &s,
                                                    const Task &t, int k0) {
        const int64_t past = (int64_t)k0 - t.border;  // the border is past all keys of a chain
        uint32_t see = below(t.pos + 1 - k0);
        if (past > -32) see &= below((int)-past);
        if (p.window > 0) {
            const int64_t out = (int64_t)t.pos + 1 - p.window - k0;  // before the window
            see &= ~below(out < 0 ? 0 : (int)(out < 32 ? out : 32)) | below(t.sinks - k0);
        }
        if (past > -32) {
            const int words = params_again().v.words;
            if (words <= 2) {
                const uint64_t m = s.bits[threadIdx.x];
                see |= past >= 64 ? 0u : (uint32_t)(past < 0 ? m << -past : m >> past);
            } else {
                const int w = (int)(past >> 5);
                const uint64_t lo = w >= 0 && w < words ? t.mask[w] : 0u;
                const uint64_t hi = w + 1 < words ? t.mask[w + 1] : 0u;
                see |= (uint32_t)((lo | hi << 32) >> (past & 31));
            }
        }
        return see & below(t.hi - k0);
    }
#else
    // Whether this lane's query row sees a position that has a page.
    __device__ static __forceinline__ bool visible(const AttendParams &p, const Task &t, int key) {
        return key <= t.pos && key >= t.lo && key < t.hi &&
               (p.window == 0 || key > t.pos - p.window);
    }
#endif
    __device__ static __forceinline__ bf16x8 widen(uint32_t a, uint32_t b) {
        const u32x4 x = {
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true))};
        return __builtin_bit_cast(bf16x8, x);
    }
    // Elements 16 ks .. 16 ks + 15 of 32 keys (rows), 8 of them for either half of
    // the wave.
    __device__ static __forceinline__ bf16x8 keys_of(const char *rows, int ks, int lane) {
        const int r = lane & 31, h = lane >> 5;
        const int f = swizzle<D, kE4m3>(r);
        if (kE4m3) {
            const i32x2 x =
                *reinterpret_cast<const i32x2 *>(rows + r * kRow + ((ks ^ f) << 4) + h * 8);
            return widen((uint32_t)x[0], (uint32_t)x[1]);
        }
        return *reinterpret_cast<const bf16x8 *>(rows + r * kRow + (((2 * ks + h) ^ f) << 4));
    }
    // V^T of 16 keys (rows from 16 kk on): elements 32 d .. 32 d + 31, and of the keys
    // 4h .. 4h + 3 and 8 + 4h .. 8 + 4h + 3 for half h, the places of their weights.
    // A row of 8 bits takes one transposing read, one of 16 two.
    static constexpr int kReads = kE4m3 ? 1 : 2;
    static constexpr int kValueReads = kReads * (D / 32);  // of 16 keys
    struct ValueAddresses {
        uint32_t at[kValueReads];  // the second read of 16 bits is kSecond bytes further
    };
    static constexpr int kSecond = 8 * kRow;
    __device__ static __forceinline__ ValueAddresses value_addresses(uint32_t base, int lane) {
        const int i16 = lane & 15, grp = (lane >> 4) & 1, h = lane >> 5;
        const int r = kE4m3 ? 8 * (i16 >> 3) + 4 * h + ((i16 >> 1) & 3) : 4 * h + (i16 >> 2);
        const int c = kE4m3 ? grp : 2 * grp + ((i16 & 3) >> 1);
        // d and e turn bits of the chunk, which the swizzle leaves to them
        const uint32_t first =
            base + (uint32_t)(r * kRow + ((c ^ swizzle<D, kE4m3>(r)) << 4) + (i16 & 1) * 8);
        ValueAddresses v;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int e = 0; e < kReads; ++e)
                v.at[d * kReads + e] = first ^ (uint32_t)(kE4m3 ? d << 5 : d << 6 | e << 5);
        return v;
    }
    // The reads are issued and waited for in one piece: as builtins they would wait
    // for every load into LDS under way (the compiler does not know which slot they
    // read), and the tiles ahead with them.
    template <int kOffset>
    __device__ static __forceinline__ void read_values(const ValueAddresses &v,
                                                       i32x2 (&x)[kValueReads]) {
        if constexpr (kE4m3 && D == 64) {
            asm volatile("ds_read_b64_tr_b8 %0, %2 offset:%c4\n\t"
                         "ds_read_b64_tr_b8 %1, %3 offset:%c4\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(x[0]), "=&v"(x[1])
                         : "v"(v.at[0]), "v"(v.at[1]), "i"(kOffset));
        } else if constexpr (kE4m3) {
            asm volatile("ds_read_b64_tr_b8 %0, %4 offset:%c8\n\t"
                         "ds_read_b64_tr_b8 %1, %5 offset:%c8\n\t"
                         "ds_read_b64_tr_b8 %2, %6 offset:%c8\n\t"
                         "ds_read_b64_tr_b8 %3, %7 offset:%c8\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
                         : "v"(v.at[0]), "v"(v.at[1]), "v"(v.at[2]), "v"(v.at[3]), "i"(kOffset));
        } else if constexpr (D == 64) {
            asm volatile("ds_read_b64_tr_b16 %0, %4 offset:%c8\n\t"
                         "ds_read_b64_tr_b16 %1, %5 offset:%c9\n\t"
                         "ds_read_b64_tr_b16 %2, %6 offset:%c8\n\t"
                         "ds_read_b64_tr_b16 %3, %7 offset:%c9\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
                         : "v"(v.at[0]), "v"(v.at[1]), "v"(v.at[2]), "v"(v.at[3]), "i"(kOffset),
                           "i"(kOffset + kSecond));
        } else {
            asm volatile("ds_read_b64_tr_b16 %0, %8 offset:%c16\n\t"
                         "ds_read_b64_tr_b16 %1, %9 offset:%c17\n\t"
                         "ds_read_b64_tr_b16 %2, %10 offset:%c16\n\t"
                         "ds_read_b64_tr_b16 %3, %11 offset:%c17\n\t"
                         "ds_read_b64_tr_b16 %4, %12 offset:%c16\n\t"
                         "ds_read_b64_tr_b16 %5, %13 offset:%c17\n\t"
                         "ds_read_b64_tr_b16 %6, %14 offset:%c16\n\t"
                         "ds_read_b64_tr_b16 %7, %15 offset:%c17\n\t"
                         "s_waitcnt lgkmcnt(0)"
                         : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]),
                           "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
                         : "v"(v.at[0]), "v"(v.at[1]), "v"(v.at[2]), "v"(v.at[3]), "v"(v.at[4]),
                           "v"(v.at[5]), "v"(v.at[6]), "v"(v.at[7]), "i"(kOffset),
                           "i"(kOffset + kSecond));
        }
    }
    __device__ static __forceinline__ bf16x8 value_of(const i32x2 (&x)[kValueReads], int d) {
        if constexpr (kE4m3) return widen((uint32_t)x[d][0], (uint32_t)x[d][1]);
        const u32x4 y = {(uint32_t)x[2 * d][0], (uint32_t)x[2 * d][1], (uint32_t)x[2 * d + 1][0],
                         (uint32_t)x[2 * d + 1][1]};
        return __builtin_bit_cast(bf16x8, y);
    }
    // The same, one operand at a time, for the scheduler to place: where the loads
    // into LDS run three tiles ahead, the last of them were issued a tile ago.
    __device__ static __forceinline__ bf16x8 value_at(const ValueAddresses &v, int kk, int d) {
        if constexpr (kE4m3) {
            const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (__attribute__((address_space(3))) i32x2 *)(uintptr_t)(v.at[d] + 16 * kk * kRow));
            return widen((uint32_t)x[0], (uint32_t)x[1]);
        } else {
            s16x4 x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                x[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(uintptr_t)(
                        v.at[2 * d + e] + 16 * kk * kRow + e * kSecond));
            return __builtin_bit_cast(bf16x8,
                                      __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
    template <int kSub, int kk>
    __device__ static __forceinline__ void add_values(const ValueAddresses &v, const bf16x8 *w,
                                                      State &st) {
        i32x2 x[kValueReads];
        read_values<16 * kk * kRow>(v, x);
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
            st.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(value_of(x, d), w[kk], st.o[d], 0, 0,
                                                              0);
        if constexpr (kk + 1 < 2 * kSub) add_values<kSub, kk + 1>(v, w, st);
    }
#if DSPARK_TREE
    // Whether a page of positions [k0, k1) is missing from the table: probe() asks for
    // the first 64 of them, hole() waits.
    struct Probe {
        int first, last, at;  // this lane's page and its entry, the last page
    };
    __device__ static __forceinline__ Probe probe(const PagedCache &c, const int32_t *table, int k0,
                                                  int k1) {
        Probe b;
        b.first = page_of(c, k0) + (threadIdx.x & (kWave - 1));
        b.last = k0 < k1 ? page_of(c, k1 - 1) : -1;
        b.at = b.first <= b.last && b.first < c.table_width ? table[b.first] : 0;
        return b;
    }
    __device__ static __forceinline__ bool hole(const PagedCache &c, const int32_t *table,
                                                const Probe &b, bool together) {
        if (!together) return true;  // looked up key by key
        bool any = b.last >= c.table_width || (b.first <= b.last && !named(c, b.at));
#pragma unroll 4
        for (int i = b.first + kWave; i <= b.last; i += kWave)
            any |= i < c.table_width && !named(c, table[i]);
        return __any(any);
    }
#else
    // Whether a page of positions [k0, k1) is missing from the table.
    __device__ static __forceinline__ bool holes(const PagedCache &c, const int32_t *table, int k0,
                                                 int k1, bool together) {
        if (!together) return true;  // looked up key by key
        const int lane = threadIdx.x & (kWave - 1);
        const int last = page_of(c, k1 - 1);
        bool any = last >= c.table_width;
#pragma unroll 4
        for (int i = page_of(c, k0) + lane; i <= last; i += kWave)
            any |= i < c.table_width && !named(c, table[i]);
        return __any(any);
    }
#endif

    // kSub times 32 keys, from key 32 * sub of a staged tile on, against the wave's
    // 32 query rows.
    template <int kSub>
    __device__ static __forceinline__ void compute(const Slots &slots, int number, int tile, int sub,
                                                   const AttendParams &p, const Task &t,
                                                   State &st, const Lds &s, int lane) {
        const int h = lane >> 5;
        const int k0 = tile * kKeys + sub * 32, k1 = k0 + kSub * 32 - 1;
#if DSPARK_TREE
        if (k0 > t.pos_max || k0 >= t.hi ||
            (k0 >= t.sinks && p.window > 0 && k1 <= t.pos_min - p.window))
            return;
        const bool whole = k1 <= t.pos_min && k1 < t.hi && !t.hole &&
                           (p.window == 0 || k0 > t.pos_max - p.window || k1 < t.sinks);
#else
        if (k0 > t.pos_max || k0 >= t.hi || k1 < t.lo ||
            (p.window > 0 && k1 <= t.pos_min - p.window))
            return;
        const bool whole = k1 <= t.pos_min && k1 < t.hi && k0 >= t.lo && !t.hole &&
                           (p.window == 0 || k0 > t.pos_max - p.window);
#endif
        // scores, transposed: keys down the registers, queries across the lanes
        f32x16 x[kSub];
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) x[i][r] = 0.f;
        // four operands are on their way from LDS behind the product at work
        constexpr int kAhead = 4, kProducts = D / 16 * kSub;
        bf16x8 a[kAhead];
        slots.pick(number, [&](const char *slot) {
            const char *kb = slot + sub * 32 * kRow;
            auto read = [&](int u) {
                a[u % kAhead] = keys_of(kb + u % kSub * 32 * kRow, u / kSub, lane);
            };
#pragma unroll
            for (int u = 0; u < kAhead; ++u) read(u);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < kProducts; ++u) {
                x[u % kSub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[u % kAhead], st.q[u / kSub],
                                                                      x[u % kSub], 0, 0, 0);
                if (u + kAhead < kProducts) read(u + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        });
        if (!whole) {
            asm volatile("");  // a branch: few tiles are masked, selects would cost all of them
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                uint32_t no = 0;
                if (t.hole)
                    no = (uint32_t)__ballot(slot_offset(params_again().a.c, t.table,
                                                        k0 + i * 32 + (lane & 31), 0) < 0);
#if DSPARK_TREE
                // the half's own bits first: a constant place for every register then
                const uint32_t bits = (seen(p, s, t, k0 + i * 32) & ~no) >> (4 * h);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    x[i][r] = bits & 1u << (8 * (r / 4) + (r & 3)) ? x[i][r] : -INFINITY;
#else
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int y = 8 * (r / 4) + 4 * h + (r & 3);
                    x[i][r] = visible(p, t, k0 + i * 32 + y) && !(no >> y & 1) ? x[i][r]
                                                                               : -INFINITY;
                }
#endif
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
        const ValueAddresses v =
            value_addresses(slots.address(number) + kHalfSlot + sub * 32 * kRow, lane);
        // the first values are read behind the exponentials
        constexpr int kVectorCrosses = 0x2 | 0x4;  // vector and scalar instructions
        if constexpr (kWide) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) a[u] = value_at(v, u / (D / 32), u % (D / 32));
            __builtin_amdgcn_sched_barrier(kVectorCrosses);
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
        if constexpr (kWide) {
#pragma unroll
            for (int u = 0; u < kProducts; ++u) {
                const int kk = u / (D / 32), d = u % (D / 32);
                st.o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[u % kAhead], w[kk], st.o[d], 0,
                                                                  0, 0);
                if (u + kAhead < kProducts)
                    a[u % kAhead] = value_at(v, (u + kAhead) / (D / 32), (u + kAhead) % (D / 32));
                __builtin_amdgcn_sched_barrier(kVectorCrosses);
            }
        } else {
            add_values<kSub, 0>(v, w, st);
        }
    }
};

template <int D, bool kE4m3, bool kWide, bool kPadded>
__global__ __launch_bounds__(kWide ? 512 : 256, 2) void attend_tile_kernel(TileParams tp) {
    using T = Tiles<D, kE4m3, kWide, kPadded>;
    using Unit = typename T::Unit;
    constexpr int kSlots = T::kSlots, kWaveLoads = T::kWaveLoads;
    constexpr int kTileThreads = T::kThreads, kTileWaves = T::kWaves;
#if DSPARK_TREE
    constexpr int kUnitTiles = kTreeUnitTiles;
#else
    constexpr int kUnitTiles = T::kUnitTiles;
#endif
    constexpr int log_rows = T::kLogRows, block_rows = 1 << log_rows;
    __shared__ typename T::Lds s;
    __shared__ __attribute__((aligned(1024))) char slot0[kSlotBytes];
    __shared__ __attribute__((aligned(1024))) char slot1[kSlotBytes];
    __shared__ __attribute__((aligned(1024))) char slot2[kWide ? kSlotBytes : 16];
    __shared__ __attribute__((aligned(1024))) char slot3[kWide ? kSlotBytes : 16];
    const typename T::Slots slots = {slot0, slot1, slot2, slot3};
    const AttendParams &p = tp.a;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = T::wave_id();
    const int G = p.Hq / p.Hkv, wgs = gridDim.x;

    // places before every request
    if (tid == 0) s.before[0] = 0;
    if ((int64_t)p.max_rows * G <= block_rows) {
        for (int b = tid; b < p.B; b += kTileThreads) {
            const Request q = load_request(p, log_rows, b);
            const int tiles = block_of<T::kKeys>(tp, log_rows, q, 0).tiles;
            s.before[b + 1] = q.M > 0 ? (uint64_t)(kUnitTiles + tiles) * p.Hkv : 0;
        }
    } else {
        for (int b = wave; b < p.B; b += kTileWaves) {
            const Request q = load_request(p, log_rows, b);
            uint64_t n = 0;
            for (int i = lane; i < q.blocks; i += kWave)
                n += kUnitTiles + block_of<T::kKeys>(tp, log_rows, q, i).tiles;
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
#if DSPARK_TREE
    // Where all requests have one block and about as many tiles (decoding and trees in
    // a window), every workgroup gets as many whole units as another and none is cut,
    // if that takes up to 30 % longer than the even division by tiles. Short units gain
    // by it: 512 of single tokens in windows of 512 and 1024 take 43 and 69 us, cut 48
    // and 74, of trees of 12 to 24 nodes 57 and 81, cut 67 and 91; on 3000 to 4000
    // positions 190 and 202, cut 193 and 219. For long ones it matters little: on 12 to
    // 16 thousand positions, the longest 1.14 times the mean, trees take 679 us, cut 696,
    // and single tokens 636, cut 620.
    bool whole_units = false;
    if ((int64_t)p.max_rows * G <= block_rows) {
        uint32_t most = 0;
        bool all = true;
        for (int b = tid; b < p.B; b += kTileThreads) {
            const uint64_t n = s.before[b + 1] - s.before[b];
            all &= n > 0;
            const uint32_t places = (uint32_t)udiv64((int64_t)n, p.Hkv);
            most = places > most ? places : most;
        }
        const uint64_t key = ((uint64_t)!__all(all) << 32) | wave_max_u64(most);
        __syncthreads();
        if (lane == 0) s.part[wave] = key;
        __syncthreads();
        uint64_t top = 0;
        for (int i = 0; i < kTileWaves; ++i) top = s.part[i] > top ? s.part[i] : top;
        const int units = p.B * p.Hkv, most_units = (units + wgs - 1) / wgs;
        const uint64_t even = (uint64_t)udiv64((int64_t)total + wgs - 1, wgs);
        whole_units = (top >> 32) == 0 && top * most_units * 10 <= even * 13;
    }
#endif
    uint64_t per = (uint64_t)udiv64((int64_t)total + wgs - 1, wgs);
    per = per < kMinTiles + kUnitTiles ? kMinTiles + kUnitTiles : per;  // so one tile at least
    // Workgroups go to the 8 XCDs in turn: each XCD takes one run of the tiles, so
    // that units of one head meet in one L2.
    int used = (int)udiv64((int64_t)(total + per - 1), (int64_t)per);
#if DSPARK_TREE
    if (whole_units) used = p.B * p.Hkv < wgs ? p.B * p.Hkv : wgs;
#endif
    const int xcd = blockIdx.x & 7, nth = blockIdx.x >> 3;
    const int share = used / 8 + (xcd < used % 8);
#if DSPARK_TREE
    Split split = {};
    if (tp.blocks == 0) {
        if (nth >= share) {
            if (tid == 0) tp.splits[blockIdx.x] = split;
            return;
        }
    } else {
        if (blockIdx.x == 0)  // units that requests with fewer rows do not have
            for (int i = tid; i < p.B * tp.blocks; i += kTileThreads) {
                const int b = i / tp.blocks;
                if (i - b * tp.blocks < load_request(p, log_rows, b).blocks) continue;
                for (int h = 0; h < p.Hkv; ++h) tp.splits[i * p.Hkv + h].parts = 0;
            }
        if (nth >= share) return;
    }
#else
    if (nth >= share) return;
#endif
    const int g = xcd * (used / 8) + (xcd < used % 8 ? xcd : used % 8) + nth;
    uint64_t start = (uint64_t)g * per;
    uint64_t end = start + per < total ? start + per : total;
#if DSPARK_TREE
    if (whole_units) {
        auto place_of = [&](int g) {
            const int u = (int)udiv64((int64_t)g * (p.B * p.Hkv), used);
            const int b = u / p.Hkv;
            if (b == p.B) return total;
            const uint64_t n = s.before[b + 1] - s.before[b];
            return s.before[b] + (uint64_t)(u - b * p.Hkv) * (uint64_t)udiv64((int64_t)n, p.Hkv);
        };
        start = place_of(g);
        end = place_of(g + 1);
    }
#endif

    // the unit of the first place, and the first tile at or after it
    Unit next;
    uint64_t cur = start;
    {
        int b = 0, hi = p.B - 1;
        while (b < hi) {
            const int mid = (b + hi) >> 1;
            if (s.before[mid + 1] <= start) b = mid + 1;
            else hi = mid;
        }
        const Request q = load_request(p, log_rows, b);
        const uint64_t in = start - s.before[b];
        const uint64_t each = (uint64_t)udiv64((int64_t)(s.before[b + 1] - s.before[b]), p.Hkv);
        const int head = (int)udiv64((int64_t)in, (int64_t)each);
        uint64_t rest = in - (uint64_t)head * each;
        int blk = 0;
        for (int i0 = 0; q.blocks > 1; i0 += kWave) {
            const int i = i0 + lane;
            const uint64_t n =
                i < q.blocks ? (uint64_t)kUnitTiles + block_of<T::kKeys>(tp, log_rows, q, i).tiles : 0;
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
        next.b = __builtin_amdgcn_readfirstlane(b);
        next.head = __builtin_amdgcn_readfirstlane(head);
        next.blk = __builtin_amdgcn_readfirstlane(blk);
        next.q = scalar_request(p, log_rows, next.b);
        next.k = block_of<T::kKeys>(tp, log_rows, next.q, next.blk);
        int place = __builtin_amdgcn_readfirstlane((int)rest) - kUnitTiles;
        if (place < 0) {
            cur -= (int64_t)place;
            place = 0;
        }
        next.tile = next.k.at(place);
        next.left = next.k.tiles - place;
    }
    auto begin_next = [&](Unit &u) {
        const TileParams tp = params_again();
        const AttendParams &p = tp.a;
        if (++u.blk == u.q.blocks) {
            u.blk = 0;
            if (++u.head == p.Hkv) {
                u.head = 0;
                do u.q = scalar_request(p, log_rows, ++u.b);
                while (u.q.blocks == 0);
            }
        }
        u.k = block_of<T::kKeys>(tp, log_rows, u.q, u.blk);
        u.tile = u.k.at(0);
        u.left = u.k.tiles;
    };

    // The stager runs three tiles ahead; past the last one it repeats it, so that
    // a fixed number of loads is always on its way.
    int64_t left = (int64_t)(end - cur);  // places from the tile to stage to the end
    typename T::Stager sg;
    T::stager(tp, sg);
    Unit ahead = next;
    T::enter(tp, sg, ahead);
    T::look_up(tp, sg, ahead.tile);
    auto stage = [&](int number, int lane) {
        T::issue(tp, sg, ahead.tile, slots, number, lane);
        const int step = ahead.left > 1 ? 1 : 1 + kUnitTiles;
        if (left > step) {
            left -= step;
            if (--ahead.left == 0) {
                begin_next(ahead);
                T::enter(tp, sg, ahead);
                T::look_up(tp, sg, ahead.tile);
            } else {
                const int tile = ahead.k.after(ahead.tile);
                const bool jump = kTree && tile != ahead.tile + 1;
                ahead.tile = tile;
                if (jump || tile - sg.batch0 == kWave) T::look_up(tp, sg, tile);
            }
        }
    };
#pragma unroll 1
    for (int i = 0; i < kSlots - 1; ++i) stage(i, lane);

    typename T::Task t;
    typename T::State st;
    int n = 0, rows = 0, qts = 1, kgs = 1, qt = 0, kg = 0, m = 0, hq = 0;
    int each = 1;  // times 32 keys of a tile for every group of waves
    int64_t row = 0;
    bool valid = false;

    // one tile: its arrival, the loads of the third after it, its products
    auto step = [&](int number) {
        // addresses are made anew for every tile: kept for all slots they would not
        // fit the registers
        int lane = threadIdx.x & (kWave - 1);
        asm volatile("" : "+v"(lane));
        const int tile = next.tile;
        const bool part = T::partial(p, t, tile);
        wait_loads<(kSlots - 2) * kWaveLoads>();
        if (part) T::scrub(s, slots, number, lane);
        asm volatile("" ::: "memory");  // no access to LDS is moved across the barrier
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // Where three tiles are on their way the next loads wait for this tile's
        // products: issued by all waves at once they hold the waves up.
        if (!kWide) stage((number + kSlots - 1) & (kSlots - 1), lane);
        if (t.active) {
            if constexpr (kWide) {
#pragma unroll 1
                for (int sub = 0; sub < T::kKeys / 32; sub += 2)
                    T::template compute<2>(slots, number, tile, sub, p, t, st, s, lane);
            } else {
#pragma unroll 1
                for (int i = 0; i < each; ++i)
                    T::template compute<1>(slots, number, tile, kg * each + i, p, t, st, s, lane);
            }
            if (part) {
                const uint64_t *bad = s.bad[number];
                uint64_t any = 0;
#pragma unroll
                for (int i = 0; i < T::kStagers * T::kRowWords; ++i) any |= bad[i];
                if (any) {
#pragma unroll 1
                    for (int i = 0; i < each; ++i)
                        T::add_bad(bad, tile, kg * each + i, p, t, st, s, lane);
                }
            }
        }
        if (kWide) stage((number + kSlots - 1) & (kSlots - 1), lane);
        next.tile = next.k.after(next.tile);
    };

    auto begin = [&]() {
        const TileParams again = params_again();
        const AttendParams &p = again.a;
        const int G = p.Hq / p.Hkv;
        const int m0 = next.blk << log_rows;
        rows = next.q.M - m0 < block_rows ? next.q.M - m0 : block_rows;
        const uint64_t rest = end - cur;
        n = (uint64_t)next.left < rest ? next.left : (int)rest;
        // 32 query rows a wave; where fewer than eight waves hold them all, the
        // others take their share of a tile's keys
        constexpr int kLogWaves = kWide ? 3 : 2;
        const int lq = kWide ? 3 : rows > 64 ? 2 : rows > 32 ? 1 : 0;
        constexpr int kLogKeys = T::kKeys == 64 ? 1 : T::kKeys == 128 ? 2 : 3;  // of 32 keys
        const int lk = kLogWaves - lq < kLogKeys ? kLogWaves - lq : kLogKeys;
        qts = 1 << lq;
        kgs = 1 << lk;
        each = 1 << (kLogKeys - lk);
        qt = wave & (qts - 1);
        kg = wave >> lq;
        const int mine = qt * 32 + (lane & 31);
        m = m0 + mine;
        valid = mine < rows;
        const int j = m / G;
        row = next.q.start + j;
        hq = next.head * G + (m - j * G);

        t.table = p.c.table + (int64_t)next.b * p.c.table_width;
        t.head_off = (int64_t)next.head * p.c.head_stride;
        t.lo = next.k.lo;
        t.hi = next.k.hi;
        t.first = next.k.first;
        t.final = next.k.final;
        t.pos = next.q.ctx + j;
        t.pos_min = next.q.ctx + (m0 + qt * 32) / G;
        const int m_last = (qt * 32 + 31 < rows - 1 ? qt * 32 + 31 : rows - 1) + m0;
        t.pos_max = next.q.ctx + m_last / G;
        t.active = kg < kgs && qt * 32 < rows;
#if DSPARK_TREE
        // queries, masks and pages are asked for together, and waited for once
        const uint16_t *src = p.q + row * p.q_row + hq * p.q_head + (lane >> 5) * 8;
        u32x4 x[D / 16];
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            x[ks] = u32x4{0u, 0u, 0u, 0u};
            const bool here = !kPadded || ks * 16 + (lane >> 5) * 8 < p.D;
            if (valid && t.active && here) x[ks] = *reinterpret_cast<const u32x4 *>(src + ks * 16);
        }
        t.border = 0x7FFFFFFF;
        t.sinks = again.v.sinks;
        int depth = j;
        uint32_t bits0 = 0, bits1 = 0;
        if (again.v.masks) {
            t.border = next.q.ctx;
            t.pos_min = next.k.first;
            t.pos_max = next.k.final;
            t.mask = again.v.masks + (valid ? row : next.q.start) * again.v.words;
            if (valid) depth = again.v.depths[row];
            if (valid && again.v.words <= 2) bits0 = t.mask[0];
            if (valid && again.v.words == 2) bits1 = t.mask[1];
        }
        const int i0 = next.k.tiles - next.left, sink = next.k.sink;
        const int s0 = i0 * T::kKeys, s1 = (i0 + n < sink ? i0 + n : sink) * T::kKeys;
        const int w0 = i0 > sink ? i0 : sink;
        const int k0 = next.k.at(w0) * T::kKeys, k1 = next.k.at(i0 + n) * T::kKeys;
        const auto in_sinks = T::probe(p.c, t.table, s0, s1 < t.hi ? s1 : t.hi);
        // the window's first tile may hold some of the sinks
        const auto in_window = T::probe(p.c, t.table, k0 > t.lo || k0 < t.sinks ? k0 : t.lo,
                                        i0 + n > sink ? (k1 < t.hi ? k1 : t.hi) : 0);
        t.pos += (depth < 0 ? 0 : depth > j ? j : depth) - j;
        s.bits[tid] = bits0 | (uint64_t)bits1 << 32;  // this lane's alone
        t.hole = T::hole(p.c, t.table, in_sinks, tp.together) ||
                 T::hole(p.c, t.table, in_window, tp.together);
#endif
        // a negative scale turns the queries' signs, none at all their values to 0
        const float scale = p.scale * p.c.k_scale;
        t.c = (scale == 0.f ? 1.f : fabsf(scale)) * kLog2e;
        const uint32_t keep = scale == 0.f ? 0u : 0xFFFFFFFFu;
        const uint32_t flip = scale < 0.f ? 0x80008000u : 0u;
        st.m = -INFINITY;
        st.l = 0.f;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) st.o[d][r] = 0.f;
#if !DSPARK_TREE
        const uint16_t *src = p.q + row * p.q_row + hq * p.q_head + (lane >> 5) * 8;
        u32x4 x[D / 16];
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            x[ks] = u32x4{0u, 0u, 0u, 0u};
            const bool here = !kPadded || ks * 16 + (lane >> 5) * 8 < p.D;
            if (valid && t.active && here) x[ks] = *reinterpret_cast<const u32x4 *>(src + ks * 16);
        }
#endif
#if !DSPARK_TREE
        const int k0 = next.tile * T::kKeys, k1 = (next.tile + n) * T::kKeys;
        t.hole = T::holes(p.c, t.table, k0 > t.lo ? k0 : t.lo, k1 < t.hi ? k1 : t.hi, tp.together);
#endif
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[ks][i] = (x[ks][i] & keep) ^ flip;
            st.q[ks] = __builtin_bit_cast(bf16x8, x[ks]);
        }
    };

    // the unit's tiles here are done: joins the waves, stores the rows or leaves
    // them for the last workgroup
    auto finish = [&]() {
        const TileParams tp = params_again();
        const AttendParams &p = tp.a;
        [[maybe_unused]] const int G = p.Hq / p.Hkv;
        st.l = half_sum(st.l);
        // the groups of keys meet, 32 elements of all rows at a time
        for (int half = kWide ? 0 : kgs / 2; half >= 1; half /= 2) {
            const bool from = t.active && kg >= half && kg < 2 * half;
            const bool to = t.active && kg < half;
            const int at = (qt + qts * (from ? kg - half : kg)) * kWave + lane;  // below kTileThreads / 2
            float a = 0.f, c = 0.f;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
                __syncthreads();
                if (from) {
                    if (d == 0) s.ml[at] = f32x2{st.m, st.l};
#pragma unroll
                    for (int r = 0; r < 16; ++r) s.join[r * (kTileThreads / 2) + at] = st.o[d][r];
                }
                __syncthreads();
                if (to) {
                    if (d == 0) {
                        const f32x2 o = s.ml[at];
                        const float top = fmaxf(st.m, o[0]);
                        a = st.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st.m - top);
                        c = o[0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(o[0] - top);
                        st.m = top;
                        st.l = st.l * a + o[1] * c;
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        st.o[d][r] = st.o[d][r] * a + s.join[r * (kTileThreads / 2) + at] * c;
                }
            }
        }
#if DSPARK_TREE
        Split *const own = tp.blocks == 0
                               ? nullptr
                               : tp.splits + (next.b * tp.blocks + next.blk) * p.Hkv + next.head;
        if (own && tid == 0 && n == next.k.tiles) own->parts = 0;
#endif
        if (n == next.k.tiles) {
            if (kg == 0 && t.active && valid) {
                const float norm = st.l > 0.f ? p.c.v_scale / st.l : 0.f;
                uint16_t *o = p.out + (row * p.Hq + hq) * (kPadded ? p.D : D) + (lane >> 5) * 4;
#pragma unroll
                for (int d = 0; d < D / 32; ++d)
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        const uint64_t y =
                            (uint64_t)pack_bf16(st.o[d][r] * norm, st.o[d][r + 1] * norm) |
                            ((uint64_t)pack_bf16(st.o[d][r + 2] * norm, st.o[d][r + 3] * norm)
                             << 32);
                        if (!kPadded || d * 32 + 2 * r < p.D)
                            *reinterpret_cast<uint64_t *>(o + d * 32 + 2 * r) = y;
                    }
            }
            return;
        }
        const uint64_t unit = cur - (uint64_t)(next.k.tiles - next.left);
        const int g0 = (int)udiv64((int64_t)unit, (int64_t)per);
        const int g1 = (int)udiv64((int64_t)(unit + next.k.tiles - 1), (int64_t)per);
        const int64_t size = slot_floats(tp.slot_rows, D);
        auto slot_of = [&](int w) { return tp.slots + size * (2 * (int64_t)w + (w == g0)); };
        const int m0 = next.blk << log_rows;
#if DSPARK_TREE
        // left for join_kernel: nothing here waits for the stores
        if (kg == 0 && t.active) {
            float *to = slot_of(g);
            if (lane < 32 && valid)
                *reinterpret_cast<f32x2 *>(to + 2 * (qt * 32 + lane)) = f32x2{st.m, st.l};
            to += 2 * tp.slot_rows + (int64_t)qt * (32 * D) + 4 * lane;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    if (valid) *reinterpret_cast<f32x4 *>(to + (d * 4 + r / 4) * (4 * kWave)) =
                        f32x4{st.o[d][r], st.o[d][r + 1], st.o[d][r + 2], st.o[d][r + 3]};
        }
        if (next.left == next.k.tiles) {
            split.parts = g1 - g0 + 1;
            split.first = g0;
            split.rows = rows;
            split.head = next.head;
            split.start = next.q.start;
            split.m0 = m0;
            if (own && tid == 0) *own = split;
        }
    };
#else
        // pairs of elements in the order of the registers, a wave's 64 pairs together
        constexpr int kPairs = D / 4;  // of a lane
        if (kg == 0 && t.active) {
            float *to = slot_of(g);
            if (lane < 32) store_coherent(to + 2 * (qt * 32 + lane), st.m, st.l);
            to += 2 * tp.slot_rows + (int64_t)qt * (32 * D) + 2 * lane;
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 2)
                    store_coherent(to + (d * 8 + r / 2) * (2 * kWave), st.o[d][r], st.o[d][r + 1]);
        }
        __builtin_amdgcn_s_waitcnt(0);  // the partial results are at the coherence point
        __syncthreads();
        if (tid == 0) {
            const unsigned old = __hip_atomic_fetch_add(tp.arrivals + g0, (unsigned)n,
                                                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            s.last = old + (unsigned)n == (unsigned)next.k.tiles;
            if (s.last)  // zero again for the next call
                __hip_atomic_store(tp.arrivals + g0, 0u, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!s.last) return;
        // A part whose row saw nothing has no maximum and holds zeros. One whose scores
        // were NaN has none either (fmaxf drops NaN), but a sum and values that are
        // NaN: no part is left out, whatever its factor.
        // First the factor of every part and row, as many rows at a time as s.join
        // holds, then the pairs of elements: 16 loads are on their way a thread,
        // two parts of eight pairs or, where there are few pairs, 16 parts of one.
        const int parts = g1 - g0 + 1;
        constexpr int kTable = 16 * (T::kWaves / 2) * kWave / 2;
        const int most = kTable / parts;  // 512 parts at most: two rows or more
        float *factor = s.join, *share = s.join + kTable;
        for (int r0 = 0; r0 < rows; r0 += most) {
            const int nr = rows - r0 < most ? rows - r0 : most;
            f32x2 ml[kTable / T::kThreads];
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kTable / T::kThreads; ++u) {
                const int i = u * T::kThreads + tid;
                ml[u] = f32x2{-INFINITY, 0.f};
                if (i < nr * parts) ml[u] = load_coherent(slot_of(g0 + i / nr) + 2 * (r0 + i % nr));
            }
#pragma unroll
            for (int u = 0; u < kTable / T::kThreads; ++u) {
                const int i = u * T::kThreads + tid;
                if (i < nr * parts) share[i] = ml[u][0];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kTable / T::kThreads; ++u) {
                const int i = u * T::kThreads + tid;
                if (i >= nr * parts) break;
                float top = -INFINITY;
                for (int w = i % nr; w < nr * parts; w += nr) top = fmaxf(top, share[w]);
                factor[i] = ml[u][0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[u][0] - top);
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kTable / T::kThreads; ++u) {
                const int i = u * T::kThreads + tid;
                if (i < nr * parts) share[i] = factor[i] * ml[u][1];
            }
            __syncthreads();
            const int items = nr * (D / 2);
            auto place = [&](int i, int &x, int64_t &at) {  // k: half, pair
                x = i % nr;
                const int k = i / nr, r = r0 + x;
                at = 2 * tp.slot_rows + (int64_t)(r >> 5) * (32 * D) + (k >> 1) * (2 * kWave) +
                     2 * ((r & 31) + 32 * (k & 1));
            };
            auto finish_pair = [&](int i, float l, f32x2 v) {
                const int x = i % nr, k = i / nr, pair = k >> 1;
                const float norm = l > 0.f ? p.c.v_scale / l : 0.f;
                const int d = pair / 8 * 32 + pair % 8 / 2 * 8 + (k & 1) * 4 + pair % 2 * 2;
                const int mm = m0 + r0 + x, jj = mm / G, hh = next.head * G + (mm - jj * G);
                if (!kPadded || d < p.D)
                    *reinterpret_cast<uint32_t *>(
                        p.out + ((int64_t)(next.q.start + jj) * p.Hq + hh) * (kPadded ? p.D : D) +
                        d) = pack_bf16(v[0] * norm, v[1] * norm);
            };
            auto sums = [&](auto pairs_at_once, auto parts_at_once) {
                constexpr int kPairs = decltype(pairs_at_once)::value;
                constexpr int kParts = decltype(parts_at_once)::value;
                for (int i0 = tid; i0 < items; i0 += T::kThreads * kPairs) {
                    int x[kPairs];
                    int64_t at[kPairs];
                    float l[kPairs];
                    f32x2 v[kPairs];
#pragma unroll
                    for (int u = 0; u < kPairs; ++u) {
                        const int i = i0 + u * T::kThreads;
                        place(i < items ? i : i0, x[u], at[u]);
                        l[u] = 0.f;
                        v[u] = f32x2{0.f, 0.f};
                    }
#pragma unroll 1
                    for (int w0 = 0; w0 < parts; w0 += kParts) {
                        f32x2 y[kParts][kPairs];
#pragma unroll
                        for (int w = 0; w < kParts; ++w)
#pragma unroll
                            for (int u = 0; u < kPairs; ++u)
                                y[w][u] = load_coherent(
                                    slot_of(g0 + (w0 + w < parts ? w0 + w : w0)) + at[u]);
#pragma unroll
                        for (int w = 0; w < kParts; ++w) {
                            if (w0 + w >= parts) break;
#pragma unroll
                            for (int u = 0; u < kPairs; ++u) {
                                const float f = factor[(w0 + w) * nr + x[u]];
                                l[u] += share[(w0 + w) * nr + x[u]];
                                v[u][0] += f * y[w][u][0];
                                v[u][1] += f * y[w][u][1];
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kPairs; ++u)
                        if (i0 + u * T::kThreads < items)
                            finish_pair(i0 + u * T::kThreads, l[u], v[u]);
                }
            };
            if (items > 2 * T::kThreads)
                sums(std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
            else
                sums(std::integral_constant<int, 1>(), std::integral_constant<int, 16>());
        }
    };
#endif

    begin();
    int done = 0;  // tiles of the unit
    for (int number = 0;; number = (number + 1) & (kSlots - 1)) {
        step(number);
        if (++done < n) continue;
        finish();
        cur += (uint64_t)(n + kUnitTiles);
        if (cur >= end) break;
        begin_next(next);
        begin();
        done = 0;
    }
    wait_loads<0>();  // nothing of this workgroup may land in LDS after it ends
#if DSPARK_TREE
    const TileParams again = params_again();
    if (tid == 0 && again.blocks == 0) again.splits[blockIdx.x] = split;
#endif
}

#if DSPARK_TREE
// Joins the parts of cut units: a workgroup takes some blocks of 32 rows by 32
// elements of a unit (every gridDim.y-th), a thread four elements of one row, eight
// parts on their way, their maximum and sums carried along. Joined by the last
// workgroup to arrive, as chains are, the parts of one tree of 60 nodes on 4000
// positions took 53 of 81 us: a tree has many rows, and few workgroups joined them all.
// A part whose row saw nothing has no maximum and holds zeros. One whose scores were
// NaN has none either, but a sum and values that are NaN: no part is left out,
// whatever its factor.
constexpr int kJoinThreads = 256;
template <int D, bool kPadded, int kAhead>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(TileParams tp) {
    const Split u = tp.splits[blockIdx.x];
    if (u.parts == 0) return;
    const AttendParams &p = tp.a;
    const int lane = threadIdx.x & (kWave - 1), r4 = threadIdx.x / kWave;
    const int64_t size = slot_floats(tp.slot_rows, D);
    const float *slots = tp.slots + size * 2 * (int64_t)u.first;
    const int G = p.Hq / p.Hkv;
    const int blocks = (u.rows + 31) / 32 * (D / 32);
    for (int i = blockIdx.y; i < blocks; i += gridDim.y) {
        const int qt = i / (D / 32), d = i % (D / 32);
        const int row = qt * 32 + (lane & 31);
        const int e = d * 32 + 8 * r4 + 4 * (lane >> 5);
        if (row >= u.rows || (kPadded && e >= p.D)) continue;
        const uint32_t at =
            2 * tp.slot_rows + qt * (32 * D) + (d * 4 + r4) * (4 * kWave) + 4 * lane;
        float top = -INFINITY, l = 0.f;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        for (int w0 = 0; w0 < u.parts; w0 += kAhead) {
            f32x2 ml[kAhead];
            f32x4 y[kAhead];
#pragma unroll
            for (int w = 0; w < kAhead; ++w) {
                // the first part lies in its workgroup's second slot
                const int n = w0 + w < u.parts ? w0 + w : w0;
                const float *x = slots + size * (2 * (int64_t)n + (n == 0));
                ml[w] = *reinterpret_cast<const f32x2 *>(x + (uint32_t)(2 * row));
                y[w] = *reinterpret_cast<const f32x4 *>(x + at);
            }
            __builtin_amdgcn_sched_barrier(0);  // all loads first
            float m1 = top;
#pragma unroll
            for (int w = 0; w < kAhead; ++w) m1 = fmaxf(m1, ml[w][0]);
            const float keep = top == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(top - m1);
            top = m1;
            l *= keep;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] *= keep;
#pragma unroll
            for (int w = 0; w < kAhead; ++w) {
                const bool one = w0 + w < u.parts;
                const float f =
                    ml[w][0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[w][0] - top);
                l += one ? f * ml[w][1] : 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] += one ? f * y[w][k] : 0.f;
            }
        }
        const float norm = l > 0.f ? p.c.v_scale / l : 0.f;
        const int mm = u.m0 + row, jj = mm / G, hh = u.head * G + (mm - jj * G);
        uint16_t *o = p.out + ((int64_t)(u.start + jj) * p.Hq + hh) * (kPadded ? p.D : D) + e;
        *reinterpret_cast<uint64_t *>(o) = (uint64_t)pack_bf16(v[0] * norm, v[1] * norm) |
                                           ((uint64_t)pack_bf16(v[2] * norm, v[3] * norm) << 32);
    }
}
#endif

static int tile_wgs(bool wide) { return device_cu_count() * (wide ? 1 : 2); }
// Calls whose requests may have over 128 query rows of a key-value head (prompts)
// take blocks of 256, eight waves of 32 rows against all keys of a tile: the keys
// are read from L2 half as often. Others share a tile's keys out to the waves. One
// kernel for both spilled its registers. Measured on either side, us in blocks of 256
// and of 128 (256 requests at 128 to 4096 with groups of 8, but for the prompts):
//   windows of 32, all whole (256 rows)     514 and 654, e4m3  534 and 604
//   windows of 64, all whole                998 and 1237       1044 and 1154
//   windows of up to 17 (136), ragged       437 and 417        524 and 359
//   windows of up to 64, ragged             628 and 625        722 and 598
//   4 prompts of 256, 1024 and 4096 rows    38, 95, 721 and 39, 103, 837
//                                    e4m3   38, 102, 752 and 31, 108, 855
//   2048 rows on 14000                      601 and 717
//     packed with 64, 256 tokens at 2000    742, 1253 and 831, 1120 (groups of 4)
// So the rule serves whole windows and prompts; where most of a call's requests have
// few rows, one of eight waves works for each, and ragged 8-bit windows pay most.
static bool tile_wide(int max_rows, int Hq, int Hkv) {
    return (int64_t)max_rows * (Hq / Hkv) > kNarrowRows;
}
static int tile_slot_rows(int max_rows, int Hq, int Hkv) {
    const int64_t m = (int64_t)max_rows * (Hq / Hkv);
    return m >= kWideRows ? kWideRows : (int)((m + 31) / 32 * 32);
}
static size_t tile_arrival_bytes() { return ((size_t)tile_wgs(false) * 4 + 255) & ~(size_t)255; }
static size_t tile_split_bytes() { return (size_t)tile_wgs(false) * sizeof(Split); }

// The head size of the tiles for heads of D, 0 where they do not serve it: a row is
// loaded 16 bytes at a time.
static int tile_head(int D, bool e4m3) {
    if (D > 128 || (e4m3 && D % 16 != 0)) return 0;
    return D > 64 ? 128 : 64;
}

[[maybe_unused]] static size_t ws_bytes(int B, int max_rows, int Hq, int Hkv, int D) {
    (void)B;
    const int head = tile_head(D, false);  // the same for either type of cache
    if (head == 0) return 256;
    auto need = [&](int rows) {
        return (size_t)2 * tile_wgs(tile_wide(rows, Hq, Hkv)) *
               (size_t)slot_floats(tile_slot_rows(rows, Hq, Hkv), head) * 4;
    };
    size_t slots = need(max_rows);
    // A call may have fewer rows, and the kernel for those twice the workgroups.
    const int narrow = kNarrowRows / (Hq / Hkv);  // the most rows it takes
    if (tile_wide(max_rows, Hq, Hkv) && narrow > 0 && need(narrow) > slots) slots = need(narrow);
    return (kZeroBytes + tile_arrival_bytes() + tile_split_bytes() + slots + 255) & ~(size_t)255;
}

template <int D, bool kE4m3>
static hipError_t launch_tiles(const AttendParams &p, const TreeView &v, void *ws, hipStream_t s) {
    TileParams tp;
    tp.a = p;
    char *at = static_cast<char *>(ws);
    tp.zeros = at;
    tp.arrivals = reinterpret_cast<unsigned *>(at + kZeroBytes);
    tp.slots = reinterpret_cast<float *>(at + kZeroBytes + tile_arrival_bytes() +
                                         tile_split_bytes());
    tp.slot_rows = tile_slot_rows(p.max_rows, p.Hq, p.Hkv);
    const int64_t item = kE4m3 ? 1 : 2;
    tp.together = p.c.page % 16 == 0 && p.c.page_stride * item < (1ll << 32) &&
                  p.c.slot_stride * item * p.c.page < (1ll << 32);
    tp.page_bytes = (uint32_t)(p.c.page_stride * item);
    tp.slot_bytes = (uint32_t)(p.c.slot_stride * item);
#if DSPARK_TREE
    tp.v = v;
    tp.splits = reinterpret_cast<Split *>(at + kZeroBytes + tile_arrival_bytes());
#endif
    for (int b = 0; b < p.B; b += kGroupRequests) {
        tp.a.B = p.B - b < kGroupRequests ? p.B - b : kGroupRequests;
        tp.a.cu = p.cu + b;
        tp.a.ctx = p.ctx + b;
        tp.a.c.table = p.c.table + (int64_t)b * p.c.table_width;
        auto go = [&](auto wide, auto padded) {
            constexpr bool kWide = decltype(wide)::value, kPadded = decltype(padded)::value;
#if DSPARK_TREE
            constexpr int kRows = 1 << Tiles<D, kE4m3, kWide, kPadded>::kLogRows;
            const int64_t most = (int64_t)p.max_rows * (p.Hq / p.Hkv);
            const int64_t units = (int64_t)tp.a.B * p.Hkv * ((most + kRows - 1) / kRows);
            const bool few = units * 4 < tile_wgs(kWide);
            const int rows = (int)(most < kRows ? most : kRows);
            tp.blocks = few ? (int)((most + kRows - 1) / kRows) : 0;
#endif
            hipLaunchKernelGGL((attend_tile_kernel<D, kE4m3, kWide, kPadded>),
                               dim3(tile_wgs(kWide)),
                               dim3(Tiles<D, kE4m3, kWide, kPadded>::kThreads), 0, s, tp);
#if DSPARK_TREE
            // Few units are cut into many parts each, of which 16 are read at once (one
            // tree of 60 nodes: 42 us, 50 with two). Many are cut in two, mostly (128
            // trees: 176 us, 195 with 16). A workgroup for every block of few units, where
            // one for every workgroup of the tiles' kernel took 36 us for that tree, 32 so.
            const int all = (rows + 31) / 32 * (D / 32);
            if (few)
                hipLaunchKernelGGL((join_kernel<D, kPadded, 16>), dim3((unsigned)units, all),
                                   dim3(kJoinThreads), 0, s, tp);
            else
                hipLaunchKernelGGL((join_kernel<D, kPadded, 2>),
                                   dim3(tile_wgs(kWide), all < 16 ? all : 16),
                                   dim3(kJoinThreads), 0, s, tp);
#endif
        };
        const std::true_type yes;
        const std::false_type no;
        if (tile_wide(p.max_rows, p.Hq, p.Hkv)) {
            if (p.D == D) go(yes, no);
            else go(yes, yes);
        } else {
            if (p.D == D) go(no, no);
            else go(no, yes);
        }
    }
    return hipGetLastError();
}

static hipError_t launch(const AttendParams &p, const TreeView &v, bool e4m3, void *ws,
                         hipStream_t s) {
    // an 8-bit cache may be aligned to 8 bytes only
    const bool aligned = (((uintptr_t)p.c.k | (uintptr_t)p.c.v) % 16 == 0) &&
                         (!e4m3 || (p.c.page_stride | p.c.head_stride | p.c.slot_stride) % 16 == 0);
    switch (aligned ? tile_head(p.D, e4m3) : 0) {
    case 128:
        return e4m3 ? launch_tiles<128, true>(p, v, ws, s) : launch_tiles<128, false>(p, v, ws, s);
    case 64:
        return e4m3 ? launch_tiles<64, true>(p, v, ws, s) : launch_tiles<64, false>(p, v, ws, s);
    }
    const dim3 grid((unsigned)p.rows, (unsigned)p.Hq);
    if (e4m3) hipLaunchKernelGGL((attend_row_kernel<true>), grid, dim3(kRowThreads), 0, s, p, v);
    else hipLaunchKernelGGL((attend_row_kernel<false>), grid, dim3(kRowThreads), 0, s, p, v);
    return hipGetLastError();
}

#if DSPARK_TREE
}  // namespace trees

hipError_t launch_tree_attention(const AttendParams &p, const TreeView &v, bool e4m3, void *ws,
                                 hipStream_t s) {
    return trees::launch(p, v, e4m3, ws, s);
}
#else
}  // namespace chains

size_t attention_ws_bytes(int B, int max_rows, int Hq, int Hkv, int D) {
    return chains::ws_bytes(B, max_rows, Hq, Hkv, D);
}

hipError_t launch_attention(const AttendParams &p, bool e4m3, void *ws, hipStream_t s) {
    return chains::launch(p, TreeView{}, e4m3, ws, s);
}
#endif

}  // namespace dspark
