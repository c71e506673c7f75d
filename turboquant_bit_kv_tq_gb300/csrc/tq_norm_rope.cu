// Norm of query and key heads with the rotation of positions.
//
//   y = x / sqrt(mean x^2 + eps) * w;  (a, b) -> (a cos p - b sin p, b cos p + a sin p)
//
// d/16 lanes hold a head, 16 elements each: for a rotated part the two pieces of 8
// whose elements (or, interleaved, whose halves) are paired, so that a rotation needs
// no exchange; elsewhere two neighbouring pieces.  A warp takes a token, 4 (d = 128) or 2
// heads at a time, and computes the token's sines once, each lane some of those that
// the lanes beside it with the same pieces need, too.  With few tokens a token's heads go
// to several warps.  Bound by memory (every element in and out once).
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
    int parts;  // warps per token
};

constexpr int kRopeThreads = 128;

// 8 elements, as they lie in memory
template <int DT>
struct RopeRaw {
    static constexpr int N = DT == TQ_DTYPE_F32 ? 2 : 1;
    uint4 w[N];
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (DT == TQ_DTYPE_F32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = p[j];
    }
    __device__ __forceinline__ void store(void* base, int64_t i) const {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + i * (DT == TQ_DTYPE_F32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = w[j];
    }
    __device__ __forceinline__ void values(float* x) const {
        if constexpr (DT == TQ_DTYPE_F32) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x[4 * j] = __uint_as_float(w[j].x), x[4 * j + 1] = __uint_as_float(w[j].y);
                x[4 * j + 2] = __uint_as_float(w[j].z), x[4 * j + 3] = __uint_as_float(w[j].w);
            }
        } else {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = DT == TQ_DTYPE_BF16 ? F8Elem::from_bf16x2(u[j]) : F8Elem::from_f16x2(u[j]);
                x[2 * j] = f.x, x[2 * j + 1] = f.y;
            }
        }
    }
};
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

// sine and cosine of position p for one pair
__device__ __forceinline__ float2 rope_turn(uint64_t p, uint64_t turns) {
    const int32_t part = (int32_t)((p * turns) >> 32);  // of a full turn, in 2^-32
    float s, c;
    sincospif((float)part * 0x1p-31f, &s, &c);
    return make_float2(s, c);
}

template <int D, int DT>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
    constexpr int LPV = D / 16, VPW = 32 / LPV;  // lanes per head, heads at a time
    constexpr int U = DT == TQ_DTYPE_F32 ? 2 : 4;  // steps whose loads are under way together
    const int lane = threadIdx.x & 31, sub = lane % LPV, slot = lane / LPV;
    const int64_t item = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = item / a.parts;
    if (t >= a.n_tokens) return;  // (whole warps)
    const int part = (int)(item - t * a.parts);
    // this warp's steps: VPW heads of q, of k or of v each
    const int nq = (a.q_heads + VPW - 1) / VPW, nk = (a.kv_heads + VPW - 1) / VPW, all = nq + (a.v ? 2 : 1) * nk;
    const int i0 = (int)((int64_t)all * part / a.parts), i1 = (int)((int64_t)all * (part + 1) / a.parts);
    // the lane's two pieces of 8
    const int rp = a.rot / 16;
    const bool turned = sub < rp;
    const int p0 = turned ? sub : 2 * sub, p1 = turned ? sub + rp : 2 * sub + 1;
    // its share of the turns: pairs VPS slot .. of the eight that its pieces need (they
    // never change, so they can be read before the previous kernel's end)
    constexpr int VPS = 8 / VPW;
    uint64_t turns[VPS] = {};
    const bool sines = rp > 0 && i0 < nq + nk;
    auto pair = [&](int i) { return a.interleaved ? 4 * (i < 4 ? p0 : p1) + (i & 3) : 8 * p0 + i; };
    if (sines && turned)
#pragma unroll
        for (int i = 0; i < VPS; ++i) turns[i] = __ldg(a.turns + pair(VPS * slot + i));
    pdl_wait();  // (the launch overlaps the previous kernel's end)

    int64_t row = t;
    if (a.rows) {
        row = a.rows[t];
        if (row < -1 || row >= a.n_rows) {
            if (lane == 0) set_error(a.err, TQ_DEVERR_CHUNK);
            row = -1;
        }
    }
    float sn[8], cs[8];
    if (sines) {
        const uint64_t p = (uint64_t)(int64_t)a.pos[t];
        float2 mine[VPS];
#pragma unroll
        for (int i = 0; i < VPS; ++i) mine[i] = rope_turn(p, turns[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sn[i] = __shfl_sync(0xffffffffu, mine[i % VPS].x, i / VPS * LPV + sub);
            cs[i] = __shfl_sync(0xffffffffu, mine[i % VPS].y, i / VPS * LPV + sub);
        }
    }

    float w[16];  // the weights of kind wk
    int wk = -1;
#pragma unroll 1
    for (int ib = i0; ib < i1; ib += U) {
        RopeRaw<DT> raw[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = ib + u, kind = i < nq ? 0 : i < nq + nk ? 1 : 2;
            const int h = (i - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * VPW + slot;
            if (i >= i1 || h >= (kind ? a.kv_heads : a.q_heads) || (kind && row < 0)) {
#pragma unroll
                for (int j = 0; j < RopeRaw<DT>::N; ++j) raw[u][0].w[j] = raw[u][1].w[j] = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            const void* src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
            const int64_t from = t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + (int64_t)h * D;
            raw[u][0].load(src, from + 8 * p0);
            raw[u][1].load(src, from + 8 * p1);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = ib + u, kind = i < nq ? 0 : i < nq + nk ? 1 : 2;
            if (i >= i1 || (kind && row < 0)) continue;  // (the same for the whole warp)
            const int h = (i - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * VPW + slot;
            const bool here = h < (kind ? a.kv_heads : a.q_heads);
            void* dst = kind == 0 ? a.qo : kind == 1 ? a.ko : a.vo;
            const int64_t to = (kind ? row : t) * (kind == 0 ? a.qo_stride : kind == 1 ? a.ko_stride : a.vo_stride) + (int64_t)h * D;
            if (kind == 2) {
                if (here) raw[u][0].store(dst, to + 8 * p0), raw[u][1].store(dst, to + 8 * p1);
                continue;
            }
            float x[16];
            raw[u][0].values(x);
            raw[u][1].values(x + 8);
            if (a.norm) {
                auto squares = [&]() {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) ss = fmaf(x[j], x[j], ss);
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
                    for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
                    for (int o = LPV / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    top = fmaxf(top, sqrtf(eps));
                    if (far && top > 0.f && top < INFINITY) {
                        const uint32_t e = __float_as_uint(top) >> 23;  // 2^(127 - e), subnormal for the largest
                        const float f = __uint_as_float(e < 254u ? (254u - max(e, 1u)) << 23 : 0x00400000u);
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] *= f;
                        eps = eps * f * f;
                    }
                    const float again = squares();  // (whole warps)
                    if (far) ss = again;
                }
                const float r = rsqrtf(fmaf(ss, 1.f / D, eps));
                const void* g = kind == 0 ? a.qw : a.kw;
                if (wk != kind) {
                    wk = kind;
                    if (g) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int at = 8 * (j ? p1 : p0);
                            if (a.w_dtype == TQ_DTYPE_F32) {
                                RopeRaw<TQ_DTYPE_F32> z;
                                z.load(g, at);
                                z.values(w + 8 * j);
                            } else if (a.w_dtype == TQ_DTYPE_BF16) {
                                RopeRaw<TQ_DTYPE_BF16> z;
                                z.load(g, at);
                                z.values(w + 8 * j);
                            } else {
                                RopeRaw<TQ_DTYPE_F16> z;
                                z.load(g, at);
                                z.values(w + 8 * j);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = 1.f;
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = x[j] * r * w[j];
            }
            if (turned) {
                auto turn = [&](int j, float& y, float& z) {
                    const float yy = y, zz = z;
                    y = fmaf(yy, cs[j], -zz * sn[j]);
                    z = fmaf(zz, cs[j], yy * sn[j]);
                };
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) turn(j, x[2 * j], x[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) turn(j, x[j], x[8 + j]);
                }
            }
            if (here) {
                rope_store8<DT>(dst, to + 8 * p0, x);
                rope_store8<DT>(dst, to + 8 * p1, x + 8);
            }
        }
    }
}

template <int D, int DT>
static tq_status launch_norm_rope(NormRopeArgs a, cudaStream_t s) {
    constexpr int VPW = 32 / (D / 16), W = kRopeThreads / 32;
    int sms = 0;
    const tq_status st = device_sms(&sms);
    if (st != TQ_OK) return st;
    // a warp per token, or as many as give every SM 16 warps
    const int64_t steps = (a.q_heads + VPW - 1) / VPW + (a.v ? 2 : 1) * (int64_t)((a.kv_heads + VPW - 1) / VPW);
    a.parts = (int)std::max<int64_t>(1, std::min<int64_t>(steps, 16 * (int64_t)sms / a.n_tokens));
    if (a.n_tokens > ((int64_t)0x7FFFFFFF - 1) * W / a.parts) return TQ_ERR_INVALID_ARG;
    const int64_t blocks = (a.n_tokens * a.parts + W - 1) / W;
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
