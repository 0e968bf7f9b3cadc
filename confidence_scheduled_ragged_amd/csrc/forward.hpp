// forward.hpp - parameters, device helpers and launches of the operators around
// the target's verify forward: append to the paged cache, attention of the
// packed rows over it, and the draw of the target's tokens (gfx950, wave64).
#pragma once

#include "common.hpp"

namespace dspark {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The paged cache as a kernel sees it: element (page, head, slot, d) of either
// pool lies at page*page_stride + head*head_stride + slot*slot_stride + d
// (elements). Slot `pos % page` of page table[b*table_width + pos / page] holds
// position pos of request b.
struct PagedCache {
    void *k, *v;
    const int32_t *table;
    int table_width, pages, page;
    uint32_t page_magic;  // pos / page = umulhi(pos, page_magic) >> page_shift (page > 1)
    int page_shift;
    int64_t page_stride, head_stride, slot_stride;
    float k_scale, v_scale;
};

// The page of a position without a division: ceil(2^(32+s) / page) with
// s = ceil(log2(page)) - 1 fits in 32 bits and is exact for positions below 2^31.
inline void set_page_size(PagedCache &c, int page) {
    c.page = page;
    c.page_magic = 0;
    c.page_shift = 0;
    if (page > 1) {
        int s = 0;
        while ((1ll << (s + 1)) < page) ++s;
        c.page_shift = s;
        const unsigned long long top = 1ull << (32 + s);
        c.page_magic = (uint32_t)((top + (unsigned)page - 1) / (unsigned)page);
    }
}
__device__ __forceinline__ int page_of(const PagedCache &c, int pos) {
    return c.page == 1 ? pos : (int)(__umulhi((uint32_t)pos, c.page_magic) >> c.page_shift);
}

// Element offset of (request row of the table, position) for one head, or -1
// when the table has no page there or names one outside the pool.
__device__ __forceinline__ int64_t slot_offset(const PagedCache &c, const int32_t *row, int pos,
                                               int head) {
    const int pg = page_of(c, pos);
    if (pg >= c.table_width) return -1;
    const int at = row[pg];
    if (at < 0 || at >= c.pages) return -1;
    return (int64_t)at * c.page_stride + (int64_t)head * c.head_stride +
           (int64_t)(pos - pg * c.page) * c.slot_stride;
}

// The request that owns packed row r, found by the calling wave (all lanes
// active): the number of entries of cu[1..B] that are at most r. B when no
// request does. Four loads are issued together, so up to 256 requests cost one
// memory round trip instead of a chain of dependent ones.
__device__ __forceinline__ int wave_request_of(const int32_t *__restrict__ cu, int B, int r) {
    const int lane = threadIdx.x & (kWave - 1);
    int b = 0;
    for (int i0 = 0; i0 < B; i0 += 4 * kWave) {
        int x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kWave + lane;
            x[u] = i < B ? cu[i + 1] : 0x7FFFFFFF;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) b += __popcll(__ballot(x[u] <= r));
    }
    return b;
}

// Two floats rounded to nearest even bf16 (one instruction on gfx950), packed.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 x = {a, b};
    const bf16x2 y = __builtin_convertvector(x, bf16x2);
    return __builtin_bit_cast(uint32_t, y);
}
// A value clamped to e4m3's range (NaN stays NaN); the conversion itself would
// turn what lies past 448 into NaN.
__device__ __forceinline__ float e4m3_clamp(float x) {
    x = x > 448.f ? 448.f : x;
    return x < -448.f ? -448.f : x;
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(a), e4m3_clamp(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_clamp(c), e4m3_clamp(d), w, true);
}

struct AppendParams {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between packed rows
    const float *cos, *sin;                // [positions, half]
    int positions, half;
    const int32_t *cu, *ctx;
    int B, rows, Hq, Hkv, D;
    PagedCache c;
    uint16_t *out;  // [rows, Hq, D]
    const int32_t *depths;  // [rows], drafted trees only
};

// Steps from a root that row j of a request stands at: never more than there are rows
// before it.
__device__ __forceinline__ int depth_of(const int32_t *depths, int64_t r, int j) {
    const int d = depths[r];
    return d < 0 ? 0 : (d > j ? j : d);
}

hipError_t launch_append_kv(const AppendParams &p, bool interleaved, bool e4m3, hipStream_t s);

struct AttendParams {
    const uint16_t *q;
    int64_t q_row, q_head;  // elements
    const int32_t *cu, *ctx;
    int B, rows, max_rows, Hq, Hkv, D, window;
    float scale;
    PagedCache c;
    uint16_t *out;  // [rows, Hq, D]
};

// What dspark_tree_attention adds: rows that see some of their request's rows
// (masks and depths, or none for a chain) and first positions that stay visible.
struct TreeView {
    const int32_t *depths;   // [rows]
    const uint32_t *masks;   // [rows, words]
    int words, sinks;
};

// Scratch of the attention kernels for valid sizes.
size_t attention_ws_bytes(int B, int max_rows, int Hq, int Hkv, int D);
hipError_t launch_attention(const AttendParams &p, bool e4m3, void *ws, hipStream_t s);
hipError_t launch_tree_attention(const AttendParams &p, const TreeView &v, bool e4m3, void *ws,
                                 hipStream_t s);

struct TreeMaskParams {
    const int32_t *parents, *cu, *ctx;  // ctx nullable
    int B, rows, max_rows, words, window, sinks;
    int32_t *depths;
    uint32_t *masks;
};
hipError_t launch_tree_masks(const TreeMaskParams &p, hipStream_t s);

struct TreeAcceptParams {
    const int32_t *choice, *tokens, *parents, *cu;
    int B, rows, max_rows, width;
    int32_t *accepted, *bonus, *path;
};
hipError_t launch_tree_accept(const TreeAcceptParams &p, hipStream_t s);

// Rows of a block table over a pool of pages; forks of some of them.
struct PoolParams {
    int32_t *table, *held, *refs;
    const int32_t *lens;
    int R, width, page, pages;
    const int32_t *src, *dst;
    int n;
    int32_t *copy_src, *copy_dst, *copy_slots, *granted;
};
hipError_t launch_resize_pages(const PoolParams &p, hipStream_t s);
hipError_t launch_fork_pages(const PoolParams &p, hipStream_t s);

// Moves of whole rows of D values in the pools of all layers; strides in bytes, also
// those of `c`, whose table the moves of a path use.
struct PageMoveParams {
    void *k, *v;
    int layers, pages, page, heads, row_bytes;
    int64_t layer_stride, page_stride, head_stride, slot_stride;
    int n;  // copies, or requests
    const int32_t *src, *dst, *slots;
    PagedCache c;
    const int32_t *path, *accepted, *ctx;
    int width;
};
hipError_t launch_copy_pages(const PageMoveParams &p, hipStream_t s);
hipError_t launch_move_kv(const PageMoveParams &p, hipStream_t s);

struct SampleParams {
    const uint16_t *logits;
    const int32_t *psrc, *cu, *tokens;
    const float *uniforms;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
    int B, gamma, V;
    int32_t *sample, *acc, *bonus;
};

hipError_t launch_sample_accept(const SampleParams &p, void *ws, hipStream_t s);

}  // namespace dspark
