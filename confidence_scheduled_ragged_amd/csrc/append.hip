// append.hip - rotary position rotation of the packed rows' queries and keys,
// and the write of keys and values into the paged cache, in one pass.
//
// For every rotated pair (x1, x2) of a query or key head at position p:
//   y1 = x1 cos(p, i) - x2 sin(p, i),   y2 = x2 cos(p, i) + x1 sin(p, i)
// in fp32, rounded once. Each input is read once and each output written once,
// so HBM bytes bound the call (and the launch, for a few rows): 11624 prompt tokens
// of 16 + 4 heads into an 8-bit cache, 134 MB, take 30 us where the tensors change
// from call to call (4.5 TB/s) and 24 us where they stay the same and partly in the
// 256 MB last-level cache (5.6 TB/s); a mixed batch of 256 requests, 49 MB, 10.5 us
// (4.6 TB/s), one row 3.2 us.
#include "forward.hpp"

namespace dspark {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ void unpack8(u32x4 a, float *x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(a[i]);
        x[2 * i + 1] = bf16_hi(a[i]);
    }
}
__device__ __forceinline__ u32x4 pack8_bf16(const float *x) {
    return u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                 pack_bf16(x[6], x[7])};
}

// Eight values to the cache at element offset `at` (16-byte or 8-byte stores).
template <bool kE4m3>
__device__ __forceinline__ void store8(void *pool, int64_t at, const float *x, float scale) {
    if (kE4m3) {
        uint32_t w[2];
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i] / scale;
        w[0] = pack_e4m3(y[0], y[1], y[2], y[3]);
        w[1] = pack_e4m3(y[4], y[5], y[6], y[7]);
        *reinterpret_cast<uint64_t *>(static_cast<uint8_t *>(pool) + at) =
            (uint64_t)w[0] | ((uint64_t)w[1] << 32);
    } else {
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(pool) + at) = pack8_bf16(x);
    }
}
template <bool kE4m3>
__device__ __forceinline__ void store1(void *pool, int64_t at, float x, float scale) {
    if (kE4m3)
        static_cast<uint8_t *>(pool)[at] = (uint8_t)pack_e4m3(x / scale, 0.f, 0.f, 0.f);
    else
        static_cast<uint16_t *>(pool)[at] = (uint16_t)pack_bf16(x, 0.f);
}

// One wave takes `heads_per` heads of a packed row at a time: with D/16 items
// of 16 elements per head, a lane keeps one item's cosines and sines in
// registers for every head it visits (the table is read once per wave and not
// once per head). An item is two groups of 8: the two halves of 8 rotated
// pairs (first half i, second half i, or adjacent pairs when interleaved), or
// 16 elements that are not rotated. `split` waves share a row.
template <bool kE4m3, bool kInterleaved>
__global__ __launch_bounds__(kAppendThreads) void append_vec_kernel(AppendParams p, int split) {
    const int lane = threadIdx.x & (kWave - 1);
    const int w = blockIdx.x * (kAppendThreads / kWave) + threadIdx.x / kWave;
    const int r = w / split, part = w - r * split;
    if (r >= p.rows) return;
    const int b = wave_request_of(p.cu, p.B, r);
    if (b >= p.B) return;
    const int j = r - p.cu[b];
    const int64_t at_pos = (int64_t)(p.ctx[b] < 0 ? 0 : p.ctx[b]) + j;
    if (j < 0 || at_pos >= p.positions) return;
    const int pos = (int)at_pos;

    const int items = p.D / 16, per = kWave / items;
    const int hl = lane / items, it = lane - hl * items;
    if (hl >= per) return;
    const int rot_items = p.half / 8;  // 16 rotated elements each
    const bool rotated = it < rot_items;
    const int e0 = rotated && !kInterleaved ? 8 * it : 16 * it;
    const int e1 = rotated && !kInterleaved ? p.half + 8 * it : e0 + 8;
    float c[8], s[8];
    if (rotated) {
        const f32x4 *cp = reinterpret_cast<const f32x4 *>(p.cos + (int64_t)pos * p.half + 8 * it);
        const f32x4 *sp = reinterpret_cast<const f32x4 *>(p.sin + (int64_t)pos * p.half + 8 * it);
        const f32x4 c0 = cp[0], c1 = cp[1], s0 = sp[0], s1 = sp[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = c0[i];
            c[4 + i] = c1[i];
            s[i] = s0[i];
            s[4 + i] = s1[i];
        }
    }
    const int64_t slot = slot_offset(p.c, p.c.table + (int64_t)b * p.c.table_width, pos, 0);
    const int heads = p.Hq + 2 * p.Hkv;
#pragma unroll 2
    for (int h = part * per + hl; h < heads; h += split * per) {
        const uint16_t *src;
        if (h < p.Hq) src = p.q + r * p.q_stride + (int64_t)h * p.D;
        else if (h < p.Hq + p.Hkv) src = p.k + r * p.k_stride + (int64_t)(h - p.Hq) * p.D;
        else src = p.v + r * p.v_stride + (int64_t)(h - p.Hq - p.Hkv) * p.D;
        const u32x4 a = *reinterpret_cast<const u32x4 *>(src + e0);
        const u32x4 d = *reinterpret_cast<const u32x4 *>(src + e1);
        float x[8], y[8];
        unpack8(a, x);
        unpack8(d, y);
        if (rotated && h < p.Hq + p.Hkv) {
            if (kInterleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x1 = x[2 * i], x2 = x[2 * i + 1];
                    x[2 * i] = x1 * c[i] - x2 * s[i];
                    x[2 * i + 1] = x2 * c[i] + x1 * s[i];
                    const float y1 = y[2 * i], y2 = y[2 * i + 1];
                    y[2 * i] = y1 * c[4 + i] - y2 * s[4 + i];
                    y[2 * i + 1] = y2 * c[4 + i] + y1 * s[4 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x1 = x[i], x2 = y[i];
                    x[i] = x1 * c[i] - x2 * s[i];
                    y[i] = x2 * c[i] + x1 * s[i];
                }
            }
        }
        if (h < p.Hq) {
            uint16_t *o = p.out + ((int64_t)r * p.Hq + h) * p.D;
            *reinterpret_cast<u32x4 *>(o + e0) = pack8_bf16(x);
            *reinterpret_cast<u32x4 *>(o + e1) = pack8_bf16(y);
        } else if (slot >= 0) {
            const bool is_k = h < p.Hq + p.Hkv;
            const int64_t at = slot + (int64_t)(h - p.Hq - (is_k ? 0 : p.Hkv)) * p.c.head_stride;
            void *pool = is_k ? p.c.k : p.c.v;
            const float scale = is_k ? p.c.k_scale : p.c.v_scale;
            store8<kE4m3>(pool, at + e0, x, scale);
            store8<kE4m3>(pool, at + e1, y, scale);
        }
    }
}

// Any head size, stride and alignment: one wave per packed row, one pair or one
// element per lane at a time (the mixed batch: 42 us).
template <bool kE4m3, bool kInterleaved>
__global__ __launch_bounds__(kAppendThreads) void append_any_kernel(AppendParams p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int r = blockIdx.x * (kAppendThreads / kWave) + threadIdx.x / kWave;
    if (r >= p.rows) return;
    const int b = wave_request_of(p.cu, p.B, r);
    if (b >= p.B) return;
    const int j = r - p.cu[b];
    const int64_t at_pos = (int64_t)(p.ctx[b] < 0 ? 0 : p.ctx[b]) + j;
    if (j < 0 || at_pos >= p.positions) return;
    const int pos = (int)at_pos;
    const int64_t slot = slot_offset(p.c, p.c.table + (int64_t)b * p.c.table_width, pos, 0);
    const int heads = p.Hq + 2 * p.Hkv, half = p.half, rest = p.D - 2 * half;
    const int per_head = half + rest;  // pairs, then single elements
    auto put = [&](int h, int e, float x) {
        if (h < p.Hq) {
            p.out[((int64_t)r * p.Hq + h) * p.D + e] = (uint16_t)pack_bf16(x, 0.f);
        } else if (slot >= 0) {
            const bool is_k = h < p.Hq + p.Hkv;
            const int64_t at =
                slot + (int64_t)(h - p.Hq - (is_k ? 0 : p.Hkv)) * p.c.head_stride + e;
            store1<kE4m3>(is_k ? p.c.k : p.c.v, at, x, is_k ? p.c.k_scale : p.c.v_scale);
        }
    };
    for (int i = lane; i < heads * per_head; i += kWave) {
        const int h = i / per_head, t = i - h * per_head;
        const uint16_t *src;
        if (h < p.Hq) src = p.q + r * p.q_stride + (int64_t)h * p.D;
        else if (h < p.Hq + p.Hkv) src = p.k + r * p.k_stride + (int64_t)(h - p.Hq) * p.D;
        else src = p.v + r * p.v_stride + (int64_t)(h - p.Hq - p.Hkv) * p.D;
        if (t >= half) {
            const int e = half + t;
            put(h, e, bf16_f32(src[e]));
            continue;
        }
        const int e0 = kInterleaved ? 2 * t : t, e1 = kInterleaved ? 2 * t + 1 : half + t;
        const float x1 = bf16_f32(src[e0]), x2 = bf16_f32(src[e1]);
        if (h < p.Hq + p.Hkv) {
            const float c = p.cos[(int64_t)pos * half + t], s = p.sin[(int64_t)pos * half + t];
            put(h, e0, x1 * c - x2 * s);
            put(h, e1, x2 * c + x1 * s);
        } else {
            put(h, e0, x1);
            put(h, e1, x2);
        }
    }
}

template <bool kE4m3, bool kInterleaved>
static hipError_t launch_append_t(const AppendParams &p, hipStream_t s) {
    const int wpb = kAppendThreads / kWave;
    const int64_t item = kE4m3 ? 1 : 2;
    // 16-byte loads and stores (8-byte stores into an 8-bit cache) where every
    // group of 8 elements is aligned for them; single elements otherwise
    bool vec = p.D % 16 == 0 && p.D <= 1024 && p.half % 8 == 0 && p.q_stride % 8 == 0 &&
               p.k_stride % 8 == 0 && p.v_stride % 8 == 0 && p.c.page_stride % 8 == 0 &&
               p.c.head_stride % 8 == 0 && p.c.slot_stride % 8 == 0;
    const void *a16[] = {p.q, p.k, p.v, p.out, p.cos, p.sin};
    for (const void *x : a16) vec = vec && (uintptr_t)x % 16 == 0;
    vec = vec && (uintptr_t)p.c.k % (8 * item) == 0 && (uintptr_t)p.c.v % (8 * item) == 0;
    if (!vec) {
        hipLaunchKernelGGL((append_any_kernel<kE4m3, kInterleaved>),
                           dim3((p.rows + wpb - 1) / wpb), dim3(kAppendThreads), 0, s, p);
        return hipGetLastError();
    }
    const int per = kWave / (p.D / 16), heads = p.Hq + 2 * p.Hkv;
    const int most = (heads + per - 1) / per;
    // waves per row: enough to fill the chip (256 CUs of 16 waves) when there are
    // few rows
    int split = 1;
    while (split < most && (int64_t)p.rows * split < 4096) split *= 2;
    if (split > most) split = most;
    const int64_t waves = (int64_t)p.rows * split;
    hipLaunchKernelGGL((append_vec_kernel<kE4m3, kInterleaved>),
                       dim3((unsigned)((waves + wpb - 1) / wpb)), dim3(kAppendThreads), 0, s, p,
                       split);
    return hipGetLastError();
}

hipError_t launch_append_kv(const AppendParams &p, bool interleaved, bool e4m3, hipStream_t s) {
    if (e4m3)
        return interleaved ? launch_append_t<true, true>(p, s) : launch_append_t<true, false>(p, s);
    return interleaved ? launch_append_t<false, true>(p, s) : launch_append_t<false, false>(p, s);
}

}  // namespace dspark
