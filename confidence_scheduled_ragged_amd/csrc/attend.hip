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

size_t attention_ws_bytes(int, int, int, int, int) { return 256; }

hipError_t launch_attention(const AttendParams &p, bool e4m3, void *ws, hipStream_t s) {
    (void)ws;
    const dim3 grid((unsigned)p.rows, (unsigned)p.Hq);
    if (e4m3) hipLaunchKernelGGL((attend_row_kernel<true>), grid, dim3(kRowThreads), 0, s, p);
    else hipLaunchKernelGGL((attend_row_kernel<false>), grid, dim3(kRowThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace dspark
