// Norm of query and key heads with the rotation of positions.
//
//   y = x / sqrt(mean x^2 + eps) * w;  (a, b) -> (a cos p - b sin p, b cos p + a sin p)
//
// d/16 lanes hold a head, 16 elements each: for a rotated part the two pieces of 8
// whose elements (or, interleaved, whose halves) are paired, so that a rotation needs
// no exchange; elsewhere two neighbouring pieces.
//
// A pair turns by F 2^-64 of a full turn a position, F = its frequency / 2 pi in
// 64-bit fixed point, so position * F modulo 2^64 is the angle, reduced without any
// rounding; its top 32 bits are as fine as fp32 sines need.

#include <algorithm>
#include <cmath>
#include <new>

#include "tq_f8.cuh"

struct tq_norm_rope_plan {
    tq_norm_rope_config cfg;
    uint32_t* err;
    const uint64_t* turns;  // [rot_dim / 2]
};

namespace tq {

struct NormRopeArgs {
    const void *q, *k, *v, *qw, *kw;
    int64_t q_stride, k_stride, v_stride;
    void *qo, *ko, *vo;
    int64_t qo_stride, ko_stride, vo_stride;
    const int32_t *pos, *rows;
    const uint64_t* turns;
    int64_t n_tokens, n_rows;
    uint32_t* err;
    float eps;
    int q_heads, kv_heads, rot, interleaved, norm, w_dtype;
};

constexpr int kRopeThreads = 128;

// 8 elements of any dtype, in fp32
template <int DT>
__device__ __forceinline__ void rope_load8(const void* base, int64_t i, float* x) {
    if constexpr (DT == TQ_DTYPE_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
        const float4 a = p[0], b = p[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = DT == TQ_DTYPE_BF16 ? F8Elem::from_bf16x2(u[j]) : F8Elem::from_f16x2(u[j]);
            x[2 * j] = f.x, x[2 * j + 1] = f.y;
        }
    }
}
template <int DT>
__device__ __forceinline__ void rope_store8(void* base, int64_t i, const float* x) {
    if constexpr (DT == TQ_DTYPE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
            make_uint4(f8_pack16(x[0], x[1], DT), f8_pack16(x[2], x[3], DT), f8_pack16(x[4], x[5], DT), f8_pack16(x[6], x[7], DT));
    }
}

template <int D, int DT>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    constexpr int LPV = D / 16;
    const int sub = threadIdx.x % LPV;
    const int heads = a.q_heads + a.kv_heads * (a.v ? 2 : 1);
    const int64_t vec = (int64_t)blockIdx.x * (kRopeThreads / LPV) + threadIdx.x / LPV;
    const int64_t t = vec / heads;
    const int h = (int)(vec - t * heads);
    pdl_wait();
    const bool here = t < a.n_tokens;
    const int kind = h < a.q_heads ? 0 : h < a.q_heads + a.kv_heads ? 1 : 2;
    int64_t row = t;
    if (here && kind && a.rows) {
        row = __ldg(a.rows + t);
        if (row < -1 || row >= a.n_rows) {
            if (sub == 0) set_error(a.err, TQ_DEVERR_CHUNK);
            row = -1;
        }
    }
    // the lane's two pieces of 8
    const int rp = a.rot / 16;
    const bool turned = sub < rp && kind < 2;
    const int p0 = sub < rp ? sub : 2 * sub, p1 = sub < rp ? sub + rp : 2 * sub + 1;
    const int hk = kind == 0 ? h : h - a.q_heads - (kind == 2 ? a.kv_heads : 0);
    const void* src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int64_t from = t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + (int64_t)hk * D;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    if (here) {
        rope_load8<DT>(src, from + 8 * p0, x);
        rope_load8<DT>(src, from + 8 * p1, x + 8);
    }
    if (a.norm && kind < 2) {
        auto squares = [&]() {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = LPV / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            return ss;
        };
        float ss = squares(), eps = a.eps;
        // Squares that leave fp32's range: once more with x 2^-e, the larger of sqrt(eps)
        // and the largest element near 1 (0, infinities and NaN stay what they are)
        const bool far = !(ss < INFINITY) || fmaf(ss, 1.f / D, eps) < 0x1p-100f;
        if (__any_sync(0xffffffffu, far)) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
            for (int o = LPV / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = fmaxf(top, sqrtf(eps));
            if (far && top > 0.f && top < INFINITY) {
                const uint32_t e = __float_as_uint(top) >> 23;  // 2^(127 - e), subnormal for the largest
                const float f = __uint_as_float(e < 254u ? (254u - max(e, 1u)) << 23 : 0x00400000u);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] *= f;
                eps = eps * f * f;
            }
            const float again = squares();  // (whole warps)
            if (far) ss = again;
        }
        const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
        const void* w = kind == 0 ? a.qw : a.kw;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= r;
        if (w) {
            float g[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = 8 * (j ? p1 : p0);
                if (a.w_dtype == TQ_DTYPE_F32) rope_load8<TQ_DTYPE_F32>(w, at, g + 8 * j);
                else if (a.w_dtype == TQ_DTYPE_BF16) rope_load8<TQ_DTYPE_BF16>(w, at, g + 8 * j);
                else rope_load8<TQ_DTYPE_F16>(w, at, g + 8 * j);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= g[i];
        }
    }
    if (here && turned) {
        const uint64_t p = (uint64_t)(int64_t)__ldg(a.pos + t);
        auto turn = [&](int pair, float& u, float& w) {
            const int32_t part = (int32_t)((p * __ldg(a.turns + pair)) >> 32);
            float c, s;
            sincospif((float)part * 0x1p-31f, &s, &c);
            const float uu = u, ww = w;
            u = fmaf(uu, c, -ww * s);
            w = fmaf(ww, c, uu * s);
        };
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn(4 * (i < 4 ? p0 : p1) + (i & 3), x[2 * i], x[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn(8 * p0 + i, x[i], x[8 + i]);
        }
    }
    if (!here || row < 0) return;
    void* dst = kind == 0 ? a.qo : kind == 1 ? a.ko : a.vo;
    const int64_t to = row * (kind == 0 ? a.qo_stride : kind == 1 ? a.ko_stride : a.vo_stride) + (int64_t)hk * D;
    rope_store8<DT>(dst, to + 8 * p0, x);
    rope_store8<DT>(dst, to + 8 * p1, x + 8);
}

template <int D, int DT>
static tq_status launch_norm_rope(const NormRopeArgs& a, cudaStream_t s) {
    const int heads = a.q_heads + a.kv_heads * (a.v ? 2 : 1);
    constexpr int VPB = kRopeThreads / (D / 16);
    if (a.n_tokens > (int64_t)0x7FFFFFFF * VPB / heads - VPB) return TQ_ERR_INVALID_ARG;
    const int64_t blocks = (a.n_tokens * heads + VPB - 1) / VPB;
    return cuda_status(launch_pdl(true, norm_rope_kernel<D, DT>, dim3((unsigned)blocks), dim3(kRopeThreads), 0, s, a));
}

static tq_status norm_rope_check(const tq_norm_rope_config& c) {
    if (c.head_dim != 128 && c.head_dim != 256) return TQ_ERR_UNSUPPORTED;
    if (c.rot_dim < 0 || c.rot_dim > c.head_dim) return TQ_ERR_INVALID_ARG;
    if (c.rot_dim % 16) return TQ_ERR_UNSUPPORTED;
    if (c.num_kv_heads < 1 || c.num_q_heads < 1 || (int64_t)c.num_q_heads + 2 * (int64_t)c.num_kv_heads > 0x7FFFFF)
        return TQ_ERR_INVALID_ARG;
    if ((c.interleaved | c.norm) & ~1) return TQ_ERR_INVALID_ARG;
    if (!(c.eps >= 0.f) || !std::isfinite(c.eps) || !(c.base > 0.0) || !std::isfinite(c.base)) return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

constexpr size_t kRopeTurnsAt = 16;

// 2^64 f / (2 pi) modulo 2^64: the quotient in two doubles, 1 / 2 pi = hi + lo
static uint64_t turns_of(double f) {
    constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    const double q = f * hi, rest = fma(f, hi, -q) + f * lo;
    const double part = q - floor(q);  // exact, in [0, 1)
    const uint64_t a = (uint64_t)(ldexp(part, 64));
    const double r = ldexp(rest, 64);
    if (!(fabs(r) < 0x1p62)) return a;  // (a frequency beyond 2^50: nothing left to keep)
    return a + (uint64_t)(int64_t)nearbyint(r);
}

}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_norm_rope_sizes(const tq_norm_rope_config* cfg, size_t* workspace_bytes) {
    if (!cfg) return TQ_ERR_INVALID_ARG;
    const tq_status st = norm_rope_check(*cfg);
    if (st != TQ_OK) return st;
    if (workspace_bytes) *workspace_bytes = kRopeTurnsAt + (size_t)cfg->rot_dim / 2 * 8;
    return TQ_OK;
}

tq_status tq_norm_rope_create(const tq_norm_rope_config* cfg, const double* inv_freq, void* workspace_dev,
                              void* stream, tq_norm_rope_plan** out) {
    if (!cfg || !workspace_dev || !out) return TQ_ERR_INVALID_ARG;
    *out = nullptr;
    const tq_status st = norm_rope_check(*cfg);
    if (st != TQ_OK) return st;
    if ((uintptr_t)workspace_dev & 15) return TQ_ERR_MISALIGNED;
    const int pairs = cfg->rot_dim / 2;
    uint64_t words[2 + 128] = {0, 0};  // the error word, then the turns
    for (int i = 0; i < pairs; ++i) {
        const double f = inv_freq ? inv_freq[i] : pow(cfg->base, -2.0 * i / cfg->rot_dim);
        if (!std::isfinite(f)) return TQ_ERR_INVALID_ARG;
        words[2 + i] = turns_of(f);
    }
    tq_norm_rope_plan* h = new (std::nothrow) tq_norm_rope_plan();
    if (!h) return TQ_ERR_INVALID_ARG;
    h->cfg = *cfg;
    h->err = static_cast<uint32_t*>(workspace_dev);
    h->turns = reinterpret_cast<const uint64_t*>(static_cast<uint8_t*>(workspace_dev) + kRopeTurnsAt);
    cudaStream_t s = (cudaStream_t)stream;
    tq_status cs = cuda_status(cudaMemcpyAsync(workspace_dev, words, kRopeTurnsAt + 8 * (size_t)pairs, cudaMemcpyHostToDevice, s));
    if (cs == TQ_OK) cs = cuda_status(cudaStreamSynchronize(s));
    if (cs != TQ_OK) {
        delete h;
        return cs;
    }
    *out = h;
    return TQ_OK;
}

tq_status tq_norm_rope_destroy(tq_norm_rope_plan* plan) {
    delete plan;
    return TQ_OK;
}

tq_status tq_norm_rope(const tq_norm_rope_plan* c, const void* q, const void* k, const void* v, int dtype,
                       int64_t q_stride, int64_t k_stride, int64_t v_stride, const void* q_weight,
                       const void* k_weight, int w_dtype, const int32_t* positions, const int32_t* kv_rows,
                       int64_t num_tokens, int64_t num_kv_rows, void* q_out, void* k_out, void* v_out,
                       int64_t q_out_stride, int64_t k_out_stride, int64_t v_out_stride, void* stream) {
    if (!c || num_tokens < 0 || num_kv_rows < 0) return TQ_ERR_INVALID_ARG;
    if (num_tokens == 0) return TQ_OK;
    if (!q || !k || !positions || !q_out || (!k_out && num_kv_rows > 0) || (!v && v_out) || (v && !v_out && num_kv_rows > 0))
        return TQ_ERR_INVALID_ARG;
    if (dtype < TQ_DTYPE_F32 || dtype > TQ_DTYPE_F16) return TQ_ERR_INVALID_ARG;
    if ((q_weight || k_weight) && (w_dtype < TQ_DTYPE_F32 || w_dtype > TQ_DTYPE_F16)) return TQ_ERR_INVALID_ARG;
    if (!kv_rows && num_kv_rows < num_tokens) return TQ_ERR_INVALID_ARG;
    const tq_norm_rope_config& g = c->cfg;
    const int64_t qr = (int64_t)g.num_q_heads * g.head_dim, kr = (int64_t)g.num_kv_heads * g.head_dim;
    if (q_stride < qr || q_out_stride < qr || k_stride < kr || k_out_stride < kr || (v && (v_stride < kr || v_out_stride < kr)))
        return TQ_ERR_INVALID_ARG;
    if (!v) v_stride = v_out_stride = 0;
    const int sz = dtype == TQ_DTYPE_F32 ? 4 : 2;
    const uintptr_t bits = (uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)k_out | (uintptr_t)v_out |
                           (uintptr_t)q_weight | (uintptr_t)k_weight |
                           (uintptr_t)((q_stride | k_stride | v_stride | q_out_stride | k_out_stride | v_out_stride) * sz);
    if ((bits & 15) || (((uintptr_t)positions | (uintptr_t)kv_rows) & 3)) return TQ_ERR_MISALIGNED;
    NormRopeArgs a;
    a.q = q, a.k = k, a.v = v;
    a.qw = q_weight, a.kw = k_weight;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.qo = q_out, a.ko = k_out, a.vo = v_out;
    a.qo_stride = q_out_stride, a.ko_stride = k_out_stride, a.vo_stride = v_out_stride;
    a.pos = positions, a.rows = kv_rows;
    a.turns = c->turns;
    a.n_tokens = num_tokens, a.n_rows = num_kv_rows;
    a.err = c->err;
    a.eps = g.eps;
    a.q_heads = g.num_q_heads, a.kv_heads = g.num_kv_heads;
    a.rot = g.rot_dim, a.interleaved = g.interleaved, a.norm = g.norm;
    a.w_dtype = w_dtype;
    cudaStream_t s = (cudaStream_t)stream;
    if (g.head_dim == 128)
        return dtype == TQ_DTYPE_F32    ? launch_norm_rope<128, TQ_DTYPE_F32>(a, s)
               : dtype == TQ_DTYPE_BF16 ? launch_norm_rope<128, TQ_DTYPE_BF16>(a, s)
                                        : launch_norm_rope<128, TQ_DTYPE_F16>(a, s);
    return dtype == TQ_DTYPE_F32    ? launch_norm_rope<256, TQ_DTYPE_F32>(a, s)
           : dtype == TQ_DTYPE_BF16 ? launch_norm_rope<256, TQ_DTYPE_BF16>(a, s)
                                    : launch_norm_rope<256, TQ_DTYPE_F16>(a, s);
}

tq_status tq_norm_rope_get_device_error(const tq_norm_rope_plan* c, uint32_t* flags, void* stream) {
    if (!c || !flags) return TQ_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    uint32_t v = 0;
    tq_status st = cuda_status(cudaMemcpyAsync(&v, c->err, 4, cudaMemcpyDeviceToHost, s));
    if (st == TQ_OK) st = cuda_status(cudaMemsetAsync(c->err, 0, 4, s));
    if (st == TQ_OK) st = cuda_status(cudaStreamSynchronize(s));
    if (st == TQ_OK) *flags = v;
    return st;
}

}  // extern "C"
