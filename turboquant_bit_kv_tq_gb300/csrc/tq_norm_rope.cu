// Norm of query and key heads with the rotation of positions.
//
//   y = x / sqrt(mean x^2 + eps) * w;  (a, b) -> (a cos p - b sin p, b cos p + a sin p)
//
// d/16 lanes hold a head, 16 elements each: for a rotated part the two pieces of 8
// whose elements (or, interleaved, whose halves) are paired, so that a rotation needs
// no exchange; elsewhere two neighbouring pieces.  Every element goes in and out once, so
// memory is the bound: 8192 rows of 32/8 heads and their values, d = 128, bf16: 34 us,
// 5.9 TB/s (87% of a plain copy), by the second of the two kernels below.
//
// Few tokens: a warp takes a token, or some of its heads, 4 (d = 128) or 2 at a time, and
// computes the token's sines once, each lane some of those that the lanes beside it with
// the same pieces need, too.  16 rows of 32/8 heads: 2.4 us, the chain of position, sine,
// product.  (The 8192 rows took 48 us so: too little under way.)
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
    int parts;  // warps (many tokens: pieces) per token
    int slice;  // heads per piece
};

constexpr int kRopeThreads = 128;

// 8 elements, as they lie in memory
template <int DT>
struct RopeRaw {
    static constexpr int N = DT == TQ_DTYPE_F32 ? 2 : 1;
    uint4 w[N];
    __device__ __forceinline__ void load(const void* base, int64_t bytes) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + bytes);
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = p[j];
    }
    __device__ __forceinline__ void store(void* base, int64_t bytes) const {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + bytes);
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = w[j];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void set(const float* x) {
        if constexpr (DT == TQ_DTYPE_F32) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                w[j] = make_uint4(__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]), __float_as_uint(x[4 * j + 2]),
                                  __float_as_uint(x[4 * j + 3]));
        } else {
            w[0] = make_uint4(f8_pack16(x[0], x[1], DT), f8_pack16(x[2], x[3], DT), f8_pack16(x[4], x[5], DT),
                              f8_pack16(x[6], x[7], DT));
        }
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
// 8 weights from element `at` on
__device__ __forceinline__ void rope_weights(const void* g, int at, int dtype, float* w) {
    if (dtype == TQ_DTYPE_F32) {
        RopeRaw<TQ_DTYPE_F32> z;
        z.load(g, at * 4);
        z.values(w);
    } else if (dtype == TQ_DTYPE_BF16) {
        RopeRaw<TQ_DTYPE_BF16> z;
        z.load(g, at * 2);
        z.values(w);
    } else {
        RopeRaw<TQ_DTYPE_F16> z;
        z.load(g, at * 2);
        z.values(w);
    }
}

// a value's sum over the d/16 lanes of a head
template <int LPV>
__device__ __forceinline__ float rope_sum(float v) {
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float rope_squares(const float (&x)[16]) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; j += 2) s[0] = fmaf(x[j], x[j], s[0]), s[1] = fmaf(x[j + 1], x[j + 1], s[1]);
    return s[0] + s[1];
}
// Squares that leave fp32's range: the mean square of x 2^-e, with x 2^-e in place of x
// and eps 4^-e added, the larger of sqrt(eps) and the largest element near 1 (0,
// infinities and NaN stay what they are).  Whole warps; `far`: this lane's head
template <int D>
__device__ __forceinline__ float rope_far(float (&x)[16], float mean, float eps, bool far) {
    constexpr int LPV = D / 16;
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
    const float ss = rope_sum<LPV>(rope_squares(x));
    return far ? fmaf(ss, 1.f / D, eps) : mean;
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

    constexpr int SZ = DT == TQ_DTYPE_F32 ? 4 : 2;
    const int64_t second = (int64_t)(p1 - p0) * 8 * SZ;  // bytes from a lane's first piece to its second
#pragma unroll 1
    for (int kind = 0, start = 0; kind < (a.v ? 3 : 2); ++kind) {
        const int heads = kind ? a.kv_heads : a.q_heads, n = kind ? nk : nq;
        const int lo = max(i0 - start, 0), hi = min(i1 - start, n);
        start += n;
        if (lo >= hi || (kind && row < 0)) continue;
        const void* in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
        void* out = kind == 0 ? a.qo : kind == 1 ? a.ko : a.vo;
        const int64_t lane_at = (int64_t)(lo * VPW + slot) * D + 8 * p0;
        const uint8_t* src = static_cast<const uint8_t*>(in) + SZ * (t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + lane_at);
        uint8_t* dst = static_cast<uint8_t*>(out) + SZ * ((kind ? row : t) * (kind == 0 ? a.qo_stride : kind == 1 ? a.ko_stride : a.vo_stride) + lane_at);
        int h = lo * VPW + slot;
        // (a, b) of a pair, times the norm's factor, becomes (fc a - gs b, gc b + fs a): weights times sines
        float fc[8], gc[8], fs[8], gs[8];
        if (kind < 2) {
            float w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = 1.f;
            const void* g = a.norm ? kind == 0 ? a.qw : a.kw : nullptr;
            if (g)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = 8 * (j ? p1 : p0);
                    rope_weights(g, at, a.w_dtype, w + 8 * j);
                }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = a.interleaved ? w[2 * j] : w[j], g2 = a.interleaved ? w[2 * j + 1] : w[8 + j];
                fc[j] = turned ? f * cs[j] : f, gc[j] = turned ? g2 * cs[j] : g2;
                fs[j] = f * sn[j], gs[j] = g2 * sn[j];
            }
        }
        // (one step at a time: the registers of a second one's loads cost more warps than they
        // gain, 9000 rows of 8/1 heads 26.2 us, 20.7)
#pragma unroll 1
        for (int i = lo; i < hi; ++i) {
            const bool here = h < heads;
            RopeRaw<DT> raw[2];
            if (here) {
                raw[0].load(src, 0);
                raw[1].load(src + second, 0);
            } else {
                raw[0].clear();
                raw[1].clear();
            }
            if (kind < 2) {
                float x[16], r = 1.f;
                raw[0].values(x);
                raw[1].values(x + 8);
                if (a.norm) {
                    const float sum = rope_sum<LPV>(rope_squares(x));
                    float mean = fmaf(sum, 1.f / D, a.eps);  // with eps
                    const bool far = !(sum < INFINITY) || mean < 0x1p-100f;
                    if (__any_sync(0xffffffffu, far)) mean = rope_far<D>(x, mean, a.eps, far);
                    r = rsqrtf(mean);
                }
                auto turn = [&](int j, float& y, float& z) {
                    const float yy = y * r, zz = z * r;  // (first: small elements may be subnormal)
                    if (turned) {
                        y = fmaf(yy, fc[j], -zz * gs[j]);
                        z = fmaf(zz, gc[j], yy * fs[j]);
                    } else {
                        y = yy * fc[j];
                        z = zz * gc[j];
                    }
                };
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) turn(j, x[2 * j], x[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) turn(j, x[j], x[8 + j]);
                }
                raw[0].set(x);
                raw[1].set(x + 8);
            }
            if (here) {
                raw[0].store(dst, 0);
                raw[1].store(dst + second, 0);
            }
            src += VPW * D * SZ;
            dst += VPW * D * SZ;
            h += VPW;
        }
    }
}

// ------------------------------------------------------------ many tokens
// Resident blocks take pieces of tokens' rows in turn (all heads of q, k and v, where they
// fit).  A piece comes into a ring in shared memory by bulk copies, is worked on in
// place, and leaves by bulk copies, so that enough bytes are under way whatever the
// warps do; v is not touched at all.  The sines of the next piece are computed beside,
// one pair per thread.  Arithmetic on pairs
// of elements (fma.rn.f32x2).
constexpr int kRopeStages = 3, kRopeBulkWarps = 4, kRopeBulkCtas = 5;
constexpr int kRopePieceBytes = 13312;  // of a stage: 5 blocks of 3 stages share an SM
// This kernel is taken from so many pieces per SM and bytes of a piece on.  32/8 heads,
// d = 128, bf16 (12 KB): 152 tokens 3.3 us here, 3.0 by the other one; 304 3.6, 3.6; 1216
// 6.6, 7.6; 4864 22.0, 27.1.  64/8 heads (2 x 10 KB): 152 3.4, 3.5; 4864 33.8, 41.2.
// Few heads: the other one wins up to about 9000 tokens of 8/1 heads (2.5 KB: 1216 4.6, 3.5;
// 4864 11.2, 10 to 11.5; 9000 21.0, 21.0; 65536 130, 137), at d = 256 (5 KB) up to about 4000
// (2432 8.5, 7.3; 4864 16.3, 18.6; 9000 26.9, 29.0; 65536 166, 190).  The rule goes by bytes
// alone: many tokens of few heads are 5 to 14% slower so.
constexpr int kRopeBulkFrom = 2, kRopeBulkLeast = 6144;

__device__ __forceinline__ uint64_t rope_pack(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 rope_unpack(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t rope_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t rope_mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void rope_bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// cosines and sines of a token's pairs
struct __align__(16) RopeSines {
    float c[128], s[128];
};

template <int D, int DT>
__global__ void __launch_bounds__(32 * kRopeBulkWarps, kRopeBulkCtas) norm_rope_bulk_kernel(const __grid_constant__ NormRopeArgs a) {
    constexpr int LPV = D / 16, VPW = 32 / LPV, SZ = DT == TQ_DTYPE_F32 ? 4 : 2, HB = D * SZ, S = kRopeStages, W = kRopeBulkWarps;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RopeSines s_sines[2];
    __shared__ __align__(16) float s_w[D];  // the keys' weights
    __shared__ uint64_t s_bars[S];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % LPV, slot = lane / LPV;
    const int all = a.q_heads + a.kv_heads * (a.v ? 2 : 1), end_k = a.q_heads + a.kv_heads;
    const int rp = a.rot / 16;
    const bool turned = sub < rp;
    const int p0 = turned ? sub : 2 * sub, p1 = turned ? sub + rp : 2 * sub + 1;
    // this block's pieces: a.slice heads of the row [q | k | v] of a token each (grid <= pieces)
    const int64_t pieces = a.n_tokens * a.parts;
    const int count = (int)((pieces - blockIdx.x + gridDim.x - 1) / gridDim.x);
    struct Piece {
        int64_t t;
        int h0, h1;  // heads of the row
    };
    // from piece to piece without a division
    const int step_t = (int)(gridDim.x / (unsigned)a.parts), step_h = (int)(gridDim.x % (unsigned)a.parts) * a.slice;
    auto next = [&](Piece& c) {
        c.t += step_t;
        c.h0 += step_h;
        if (c.h0 >= a.parts * a.slice) c.h0 -= a.parts * a.slice, ++c.t;
        c.h1 = min(c.h0 + a.slice, all);
    };
    Piece c;  // the piece worked on
    c.t = blockIdx.x / (unsigned)a.parts;
    c.h0 = (int)(blockIdx.x % (unsigned)a.parts) * a.slice;
    c.h1 = min(c.h0 + a.slice, all);
    Piece ahead = c, coming = c;  // the next to be fetched (thread 0), the next to be worked on
    const uint64_t turns = tid < a.rot / 2 ? __ldg(a.turns + tid) : 0;  // (they never change)
    const uint32_t bars = smem_u32(s_bars);
    if (tid == 0) {
        for (int i = 0; i < S; ++i) mbar_init(bars + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();  // (the launch overlaps the previous kernel's end)

    // the parts of a piece in q, in k and in v: `copy(kind, first head of it, heads, byte in the piece)`
    auto parts = [&](const Piece& c, auto copy) {
        if (c.h0 < a.q_heads) copy(0, c.h0, min(c.h1, a.q_heads) - c.h0, 0);
        const int k0 = max(c.h0, a.q_heads), k1 = min(c.h1, end_k);
        if (k0 < k1) copy(1, k0 - a.q_heads, k1 - k0, (k0 - c.h0) * HB);
        const int v0 = max(c.h0, end_k);
        if (v0 < c.h1) copy(2, v0 - end_k, c.h1 - v0, (v0 - c.h0) * HB);
    };
    // thread 0: the next piece, k, into stage k % S
    auto fetch = [&](int k) {
        const uint32_t bar = bars + 8 * (k % S), to = smem_u32(ring) + (k % S) * (a.slice * HB);
        mbar_expect_tx(bar, (ahead.h1 - ahead.h0) * HB);
        parts(ahead, [&](int kind, int h, int n, int at) {
            const void* in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
            const int64_t stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
            bulk_copy(to + at, static_cast<const uint8_t*>(in) + ahead.t * stride * SZ + (int64_t)h * HB, n * HB, bar);
        });
        next(ahead);
    };
    int fetched = min(count, S - 1), waited = 0;
    if (tid == 0)
        for (int k = 0; k < fetched; ++k) fetch(k);
    for (int i = 8 * tid; i < D; i += 256 * W) {
        float z[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        if (a.kw) rope_weights(a.kw, i, a.w_dtype, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) s_w[i + j] = z[j];
    }
    uint64_t wq[8];  // the queries', of the lane's elements
    {
        float z[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = 1.f;
        if (a.qw) rope_weights(a.qw, 8 * p0, a.w_dtype, z), rope_weights(a.qw, 8 * p1, a.w_dtype, z + 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) wq[j] = rope_pack(z[2 * j], z[2 * j + 1]);
    }
    auto sines = [&](int k, int p) {
        if (tid >= a.rot / 2) return;
        const float2 t = rope_turn((uint64_t)(int64_t)p, turns);
        RopeSines& o = s_sines[k & 1];
        o.s[tid] = t.x, o.c[tid] = t.y;
    };
    sines(0, a.pos[c.t]);
    int64_t row = a.rows ? a.rows[c.t] : c.t;
    next(coming);
    int pos = count > 1 ? a.pos[coming.t] : 0;
    __syncthreads();

    bool dead = false;
    for (int k = 0; k < count; ++k) {
        const int stage = k % S;
        if (!dead) dead = !mbar_wait(bars + 8 * stage, (k / S) & 1, a.err);
        if (!dead) waited = k + 1;
        const int64_t next_row = k + 1 < count ? a.rows ? a.rows[coming.t] : coming.t : 0;
        uint8_t* base = ring + stage * (a.slice * HB);
        const RopeSines& sc = s_sines[k & 1];
        uint64_t cs[4] = {}, sn[4] = {};  // the lane's sines (interleaved: one of a pair in each)
        if (turned) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int pr = a.interleaved ? 4 * (j < 2 ? p0 : p1) + 2 * (j & 1) : 8 * p0 + 2 * j;
                cs[j] = *reinterpret_cast<const uint64_t*>(sc.c + pr);
                sn[j] = *reinterpret_cast<const uint64_t*>(sc.s + pr);
            }
        }
        // VPW heads from h on, with the lane's weights in pairs
        auto work = [&](int h, int top, auto weight) {
            const bool here = h + slot < top;
            uint8_t* at = base + ((here ? h + slot : h) - c.h0) * HB;
            RopeRaw<DT> raw[2];
            raw[0].load(at, 8 * p0 * SZ);
            raw[1].load(at, 8 * p1 * SZ);
            float x[16];
            raw[0].values(x);
            raw[1].values(x + 8);
            if (a.norm) {
                uint64_t q[2] = {0, 0};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint64_t z = rope_pack(x[2 * j], x[2 * j + 1]);
                    q[j & 1] = rope_fma2(z, z, q[j & 1]);
                }
                const float2 q0 = rope_unpack(q[0]), q1 = rope_unpack(q[1]);
                const float sum = rope_sum<LPV>((q0.x + q0.y) + (q1.x + q1.y));
                float mean = fmaf(sum, 1.f / D, a.eps);
                const bool far = !(sum < INFINITY) || mean < 0x1p-100f;
                if (__any_sync(0xffffffffu, far)) mean = rope_far<D>(x, mean, a.eps, far);
                const float r = rsqrtf(mean);
                const uint64_t rr = rope_pack(r, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 y = rope_unpack(rope_mul2(rope_mul2(rope_pack(x[2 * j], x[2 * j + 1]), rr), weight(j)));
                    x[2 * j] = y.x, x[2 * j + 1] = y.y;
                }
            }
            if (turned) {
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 cc = rope_unpack(cs[j / 2]), ss = rope_unpack(sn[j / 2]);
                        const float y = x[2 * j], z = x[2 * j + 1], co = j & 1 ? cc.y : cc.x, si = j & 1 ? ss.y : ss.x;
                        x[2 * j] = fmaf(y, co, -z * si);
                        x[2 * j + 1] = fmaf(z, co, y * si);
                    }
                } else {
                    const uint64_t minus = rope_pack(-1.f, -1.f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t y = rope_pack(x[2 * j], x[2 * j + 1]), z = rope_pack(x[8 + 2 * j], x[9 + 2 * j]);
                        const float2 u = rope_unpack(rope_fma2(rope_mul2(z, sn[j]), minus, rope_mul2(y, cs[j])));
                        const float2 v = rope_unpack(rope_fma2(z, cs[j], rope_mul2(y, sn[j])));
                        x[2 * j] = u.x, x[2 * j + 1] = u.y, x[8 + 2 * j] = v.x, x[9 + 2 * j] = v.y;
                    }
                }
            }
            raw[0].set(x);
            raw[1].set(x + 8);
            if (here) {
                raw[0].store(at, 8 * p0 * SZ);
                raw[1].store(at, 8 * p1 * SZ);
            }
        };
        // the piece's query heads, then its key heads; both in turn to the warps, the last first
        const int qe = min(c.h1, a.q_heads), ks = max(c.h0, a.q_heads), ke = min(c.h1, end_k);
        int h = c.h0 + (W - 1 - warp) * VPW;
        for (; h < qe; h += W * VPW) work(h, qe, [&](int j) { return wq[j]; });
        // (a step further for each of the warps: h - W VPW was this warp's last of the query heads)
        if (c.h0 < qe) h = ks + (h - c.h0 - (qe - c.h0 + VPW - 1) / VPW * VPW);
        for (; h < ke; h += W * VPW)
            work(h, ke, [&](int j) { return *reinterpret_cast<const uint64_t*>(&s_w[8 * (j < 4 ? p0 : p1) + 2 * (j & 3)]); });
        if (k + 1 < count) {
            sines(k + 1, pos);
            Piece after = coming;
            next(after);
            if (k + 2 < count) pos = a.pos[after.t];
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();  // the piece's heads and the next one's sines are written
        if (tid == 0) {
            const uint32_t from = smem_u32(base);
            if (row < -1 || (a.rows && row >= a.n_rows)) {
                if (c.h1 > a.q_heads) set_error(a.err, TQ_DEVERR_CHUNK);
                row = -1;
            }
            if (!dead)
                parts(c, [&](int kind, int h, int n, int at) {
                    if (kind && row < 0) return;
                    void* out = kind == 0 ? a.qo : kind == 1 ? a.ko : a.vo;
                    const int64_t stride = kind == 0 ? a.qo_stride : kind == 1 ? a.ko_stride : a.vo_stride;
                    rope_bulk_store(static_cast<uint8_t*>(out) + (kind ? row : c.t) * stride * SZ + (int64_t)h * HB, from + at, n * HB);
                });
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            // the stage of the piece before this one is free once its heads have left
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            if (!dead && k + S - 1 < count) fetch(k + S - 1), ++fetched;
        }
        row = next_row;
        c = coming;
        next(coming);
    }
    if (tid == 0) {
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        // after a wait that gave up: copies still in flight land before the block ends
        for (; dead && waited < fetched; ++waited) mbar_wait(bars + 8 * (waited % S), (waited / S) & 1, a.err);
    }
}

template <int D, int DT>
static tq_status launch_norm_rope(NormRopeArgs a, cudaStream_t s) {
    constexpr int VPW = 32 / (D / 16), W = kRopeThreads / 32, HB = D * (DT == TQ_DTYPE_F32 ? 4 : 2);
    int sms = 0;
    tq_status st = device_sms(&sms);
    if (st != TQ_OK) return st;
    if (a.n_tokens > (int64_t)1 << 40) return TQ_ERR_INVALID_ARG;
    // pieces of a token's heads that let kRopeBulkCtas rings share an SM
    const int64_t heads = a.q_heads + (int64_t)a.kv_heads * (a.v ? 2 : 1);
    constexpr int most = kRopePieceBytes / HB / VPW * VPW;
    const int64_t parts = (heads + most - 1) / most;
    a.slice = (int)(((heads + parts - 1) / parts + VPW - 1) / VPW * VPW);
    if (a.n_tokens * parts >= kRopeBulkFrom * (int64_t)sms && a.slice * HB >= kRopeBulkLeast) {
        st = ensure_dynamic_smem((const void*)norm_rope_bulk_kernel<D, DT>, kRopeStages * kRopePieceBytes, "norm_rope_bulk_kernel");
        if (st != TQ_OK) return st;
        a.parts = (int)((heads + a.slice - 1) / a.slice);
        const int64_t grid = std::min<int64_t>(a.n_tokens * a.parts, (int64_t)sms * kRopeBulkCtas);
        return cuda_status(launch_pdl(true, norm_rope_bulk_kernel<D, DT>, dim3((unsigned)grid), dim3(32 * kRopeBulkWarps),
                                      (size_t)kRopeStages * a.slice * HB, s, a));
    }
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

// 2^64 f / (2 pi) modulo 2^64, to the nearest: the quotient in two doubles, 1 / 2 pi = hi +
// lo.  Of the magnitude, negated at the end: of a small negative quotient the part
// above its floor would be rounded to 53 bits, or to 1.
static uint64_t turns_of(double f) {
    constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
    const double m = fabs(f), q = m * hi, rest = fma(m, hi, -q) + m * lo;
    const double units = ldexp(q - floor(q), 64), whole = floor(units);  // exact, in [0, 2^64)
    const double below = (units - whole) + ldexp(rest, 64);
    uint64_t a = (uint64_t)whole;
    if (fabs(below) < 0x1p62) a += (uint64_t)(int64_t)nearbyint(below);  // (a frequency beyond 2^50: nothing left to keep)
    return f < 0.0 ? 0 - a : a;
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
    // in place means row by row in place
    if (num_tokens > 1 && ((q_out == q && q_out_stride != q_stride) ||
                           (!kv_rows && ((k_out == k && k_out_stride != k_stride) || (v && v_out == v && v_out_stride != v_stride)))))
        return TQ_ERR_INVALID_ARG;
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
