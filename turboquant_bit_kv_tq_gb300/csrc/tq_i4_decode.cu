// Decode attention over the 4-bit cache: the plain form of the kernel.
//
// One block per (sequence, query head); its warps take every fourth token, a lane d/32
// coordinates.  With x the scale of a vector, s_t = scale log2(e) <q, k_t>,
// out = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m), m the running maximum.

#include "tq_i4.cuh"

namespace tq {

struct I4DecodeArgs {
    const void* q;
    int64_t q_stride;
    const uint8_t* cache;
    const int32_t *table, *lens;
    void* out;
    uint32_t* err;
    int64_t num_blocks;
    float scale_log2e;
    int q_dtype, out_dtype;
    int heads, q_heads, group, max_blocks;
};

constexpr int kI4Warps = 4;

__device__ __forceinline__ float i4_element(const void* p, int64_t i, int dtype) {
    if (dtype == TQ_DTYPE_F32) return __ldg(static_cast<const float*>(p) + i);
    if (dtype == TQ_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

template <int D>
__global__ void __launch_bounds__(32 * kI4Warps) i4_decode_kernel(I4DecodeArgs a) {
    constexpr int E = D / 32;
    __shared__ float s_m[kI4Warps];
    __shared__ double s_l[kI4Warps], s_o[kI4Warps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / a.q_heads, qh = blockIdx.x % a.q_heads, h = qh / a.group;
    int len = __ldg(a.lens + b);
    if (len < 0 || len > a.max_blocks * 16) {
        if (threadIdx.x == 0) set_error(a.err, TQ_DEVERR_SEQLEN);
        len = max(0, min(len, a.max_blocks * 16));
    }
    // (sums in 64 bits: values near the ends of fp32's range)
    float q[E], m = -INFINITY;
    double o[E], l = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = i4_element(a.q, (int64_t)b * a.q_stride + (int64_t)qh * D + E * lane + i, a.q_dtype);
        o[i] = 0;
    }
    auto load = [&](const uint8_t* page, int row, int which, float (&x)[E]) {
        const uint8_t* c = page + which * 8 * D + row * (D / 2) + E / 2 * lane;
        const float sc = i4_scale(__ldg(page + i4_scales_at(D) + which * D + row * (D / 16) + E * lane / 16)) *
                         f8_scale(__ldg(page + i4_exps_at(D) + 16 * which + row));
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = (float)((int)((__ldg(c + i / 2) >> (4 * (i & 1))) & 15) - 8) * sc;
    };
    for (int t = warp; t < len; t += kI4Warps) {
        const int blk = __ldg(a.table + (int64_t)b * a.max_blocks + (t >> 4));
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) set_error(a.err, TQ_DEVERR_BLOCK);
            continue;
        }
        const uint8_t* page = a.cache + ((int64_t)blk * a.heads + h) * i4_page_bytes(D);
        float x[E], s = 0.f;
        load(page, t & 15, 0, x);
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(q[i], x[i], s);
        s = warp_sum(s) * a.scale_log2e;
        const float top = fmaxf(m, s), was = m == -INFINITY ? 0.f : exp2f(m - top), p = exp2f(s - top);
        load(page, t & 15, 1, x);
        l = l * was + p;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * was + (double)p * x[i];
        m = top;
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int i = 0; i < E; ++i) s_o[warp][E * lane + i] = o[i];
    __syncthreads();
    float top = -INFINITY, f[kI4Warps];
    double sum = 0;
    for (int w = 0; w < kI4Warps; ++w) top = fmaxf(top, s_m[w]);
    for (int w = 0; w < kI4Warps; ++w) {
        f[w] = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - top);
        sum += s_l[w] * f[w];
    }
    for (int i = 2 * threadIdx.x; i < D; i += 64 * kI4Warps) {
        double x = 0, y = 0;
        for (int w = 0; w < kI4Warps; ++w) x += s_o[w][i] * f[w], y += s_o[w][i + 1] * f[w];
        if (sum != 0) x /= sum, y /= sum;
        f8_store2(a.out, (int64_t)blockIdx.x * D + i, (float)x, (float)y, a.out_dtype);
    }
}

}  // namespace tq

using namespace tq;

extern "C" tq_status tq_i4_decode_attention(const tq_i4_cache* c, const void* q, int q_dtype, int64_t q_stride,
                                            const void* cache_buf, const int32_t* block_table,
                                            const int32_t* seq_lens, float scale, int batch, void* out,
                                            int out_dtype, void* stream) {
    if (!c || !q || !cache_buf || !block_table || !seq_lens || !out) return TQ_ERR_INVALID_ARG;
    if (batch < 1 || batch > c->cfg.max_batch) return TQ_ERR_INVALID_ARG;
    if (q_dtype < TQ_DTYPE_F32 || q_dtype > TQ_DTYPE_F16 || out_dtype < TQ_DTYPE_F32 || out_dtype > TQ_DTYPE_F16)
        return TQ_ERR_INVALID_ARG;
    const int d = c->cfg.head_dim;
    if (q_stride < (int64_t)c->cfg.num_q_heads * d) return TQ_ERR_INVALID_ARG;
    const int qs = q_dtype == TQ_DTYPE_F32 ? 4 : 2;
    if (((uintptr_t)q | (uintptr_t)(q_stride * qs) | (uintptr_t)cache_buf | (uintptr_t)out) & 15) return TQ_ERR_MISALIGNED;
    I4DecodeArgs a;
    a.q = q;
    a.q_stride = q_stride;
    a.cache = static_cast<const uint8_t*>(cache_buf);
    a.table = block_table;
    a.lens = seq_lens;
    a.out = out;
    a.err = c->err;
    a.num_blocks = c->cfg.num_blocks;
    a.scale_log2e = (scale > 0.f ? scale : 1.0f / sqrtf((float)d)) * 1.4426950408889634f;
    a.q_dtype = q_dtype;
    a.out_dtype = out_dtype;
    a.heads = c->cfg.num_kv_heads;
    a.q_heads = c->cfg.num_q_heads;
    a.group = c->cfg.num_q_heads / c->cfg.num_kv_heads;
    a.max_blocks = c->cfg.max_blocks_per_seq;
    cudaStream_t s = (cudaStream_t)stream;
    const dim3 grid((unsigned)batch * (unsigned)c->cfg.num_q_heads);
    return d == 128 ? cuda_status(launch_pdl(false, i4_decode_kernel<128>, grid, dim3(32 * kI4Warps), 0, s, a))
                    : cuda_status(launch_pdl(false, i4_decode_kernel<256>, grid, dim3(32 * kI4Warps), 0, s, a));
}
