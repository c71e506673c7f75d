// Decode attention over the 8-bit cache.
//
// With k8, v8 the codes, 2^ek, 2^ev the vectors' scales and c = scale * log2(e):
//   s_t = c <q, k8_t> 2^ek_t             (log2 units)
//   l   = sum_t 2^(s_t - r)              r, r': references of the sums, moved
//   o   = sum_t 2^(s_t + ev_t - r') v8_t  when a score passes them by 2^12
//   out = o / l * 2^(r' - r)
// The value scale goes into the exponent of the weight, with a reference of its
// own, so no weight over- or underflows whatever the scales are.
//
// Bound by memory (2 d + 2 bytes per token and KV head).  All pages of all
// sequences, in the order (sequence, KV head, page), are dealt out evenly to a
// fixed grid of resident blocks; a block's run is cut into segments of one
// (sequence, KV head) each.  The warps of a block take steps of 256/d pages of a
// segment in turn; each warp keeps a ring of steps in flight with cp.async,
// which puts the rows where the tensor-core operands read them without bank
// conflicts, and prefetches across segments.  Products per 16 tokens:
//   S^T[tokens x heads] = K Q^T     mma.m16n8k16, A = codes as fp16 (exact)
//   O^T[d x heads] += V^T P^T       A = pairs of value codes, B = the weights
// so a KV head's query heads (8 or 16 columns) share every page, and tokens and
// coordinates fill the 16 rows: a group of 8 heads wastes nothing.  (tcgen05
// would want 128 rows of operands in shared memory, written back after the
// conversion; mma.sync takes the converted codes from registers and runs at
// about a third of its rate here.)
// A segment that is a whole (sequence, KV head) is written out; the others go
// to the workspace, and the last block to arrive joins them in block order.

#include <algorithm>

#include "tq_f8.cuh"

namespace tq {

struct F8DecodeArgs {
    const void* q;
    int64_t q_stride;
    const uint8_t* cache;
    const int32_t *table, *lens;
    void* out;
    uint32_t *err, *cnt;
    float *part, *meta;
    int64_t num_blocks;
    float scale_log2e;
    int q_dtype, out_dtype;
    int batch, heads, q_heads, group, nhg, hp, max_blocks;
};

constexpr int kF8Warps = 4;
constexpr int kF8Threads = 32 * kF8Warps;
// weights are kept below 2^kF8Slack and the reference is set so that the
// largest is 2^kF8Head: small weights stay normal fp16 numbers further down
constexpr float kF8Slack = 12.f, kF8Head = 4.f;

__device__ __forceinline__ float f8_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void f8_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ uint32_t f8_transpose(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t f8_pack_f16(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// remainders of (x, y) after the fp16 pair `hi`
__device__ __forceinline__ uint32_t f8_pack_rest(float x, float y, uint32_t hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return f8_pack_f16(x - f.x, y - f.y);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int D, int NT, bool PREC>
struct F8Cfg {
    static constexpr int PP = 256 / D;                 // pages per step
    static constexpr int PAGE = f8_page_bytes(D);
    static constexpr int STEP = PP * PAGE;             // bytes of a ring stage
    static constexpr int STAGES = 3;
    static constexpr int HEADS = 8 * NT;
    static constexpr int QF = (D / 16) * NT * 32 * 8 * (PREC ? 2 : 1);
    static constexpr int BUF_LD = D + 8;               // head stride of the merge buffer, in floats
    static constexpr int off_q = kF8Warps * STAGES * STEP;
    // the merge buffer takes the query operands' place: it is written once
    // every warp is through with the segment's scores
    static constexpr int off_buf = off_q;
    static constexpr int BUF = HEADS * BUF_LD * 4;
    static constexpr int off_cq = off_q + (QF > BUF ? QF : BUF);
    static constexpr int off_ref = off_cq + HEADS * 4;             // [warps][HEADS][3] r, r', l
    static constexpr int off_info = off_ref + kF8Warps * HEADS * 3 * 4;  // [warps][STAGES][PP] valid tokens
    static constexpr int total = off_info + kF8Warps * STAGES * PP * 4;
    static constexpr int CTAS = total + 1024 <= 233472 / 2 ? 2 : 1;  // per SM
};

__device__ __forceinline__ int f8_seq_pages(const F8DecodeArgs& a, int b) {
    const int len = __ldg(a.lens + b), cap = a.max_blocks * 16;
    return (max(0, min(len, cap)) + 15) >> 4;
}

// A position in the order (sequence, KV head and head group, page) and the
// pages left of a block's run.
struct F8Walk {
    int b, j, p, np;
    int64_t left;
};
struct F8Seg {
    int b, j, p0, p1, np;
};
__device__ __forceinline__ F8Seg f8_next(const F8DecodeArgs& a, F8Walk& w, int nj) {
    F8Seg s;
    s.b = w.b;
    s.j = w.j;
    s.p0 = w.p;
    s.np = w.np;
    const int n = (int)min((int64_t)(w.np - w.p), w.left);
    s.p1 = w.p + n;
    w.left -= n;
    w.p = 0;
    if (++w.j == nj) {
        w.j = 0;
        w.np = 0;
        while (w.left > 0 && w.np == 0 && ++w.b < a.batch) w.np = f8_seq_pages(a, w.b);
    }
    return s;
}

template <int D, int NT, bool PREC>
__global__ void __launch_bounds__(kF8Threads, 2) f8_decode_kernel(F8DecodeArgs a) {
    using C = F8Cfg<D, NT, PREC>;
    constexpr int S = C::STAGES, PP = C::PP, W = kF8Warps, HEADS = C::HEADS;
    extern __shared__ __align__(16) uint8_t smem[];
    uint2* qf = reinterpret_cast<uint2*>(smem + C::off_q);
    float* buf = reinterpret_cast<float*>(smem + C::off_buf);
    float* cq = reinterpret_cast<float*>(smem + C::off_cq);
    float* ref = reinterpret_cast<float*>(smem + C::off_ref);
    __shared__ long long s_scan[kF8Threads / 32 + 1], s_units[kF8Threads / 32];
    __shared__ long long s_base;
    __shared__ int s_b, s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int nj = a.heads * a.nhg;
    uint8_t* ring = smem + warp * (S * C::STEP);
    int* info = reinterpret_cast<int*>(smem + C::off_info) + warp * S * PP;

    // ---- the run of this block: totals, and the sequence its run starts in
    const int per = (a.batch + kF8Threads - 1) / kF8Threads;
    const int bt0 = min(a.batch, tid * per), bt1 = min(a.batch, bt0 + per);
    long long mine = 0, some = 0;
    for (int b = bt0; b < bt1; ++b) {
        const int len = __ldg(a.lens + b);
        if (len < 0 || len > a.max_blocks * 16) set_error(a.err, TQ_DEVERR_SEQLEN);
        const int np = f8_seq_pages(a, b);
        mine += np;
        some += np > 0;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
        some += __shfl_xor_sync(0xffffffffu, some, o);
    }
    if (lane == 31) s_scan[warp] = incl;
    if (lane == 0) s_units[warp] = some;
    if (tid == 0) s_b = -1;
    __syncthreads();
    long long before = incl - mine, total = 0, units = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        before += w < warp ? s_scan[w] : 0;
        total += s_scan[w];
        units += s_units[w];
    }
    before *= nj;
    total *= nj;
    units *= nj;
    // blocks that get a run: every one, unless it would be shorter than a
    // step of each warp (then as many as there are (sequence, KV head)s, at least)
    const long long N =
        max(1ll, min((long long)gridDim.x, max(units, (total + W * PP - 1) / (W * PP))));
    const long long u0 = min(total, (long long)blockIdx.x * total / N);
    const long long u1 = blockIdx.x < N ? ((long long)blockIdx.x + 1) * total / N : u0;
    if (u0 < u1 && before <= u0 && u0 < before + mine * nj) {
        long long at = before;
        for (int b = bt0; b < bt1; ++b) {
            const long long n = (long long)f8_seq_pages(a, b) * nj;
            if (u0 < at + n) {
                s_b = b;
                s_base = at;
                break;
            }
            at += n;
        }
    }
    // sequences without a token: their rows are zero
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        if (f8_seq_pages(a, b) > 0) continue;
        for (int i = tid; i < a.q_heads * D / 2; i += kF8Threads)
            f8_store2(a.out, (int64_t)b * a.q_heads * D + 2 * i, 0.f, 0.f, a.out_dtype);
    }
    __syncthreads();
    if (u0 >= u1) return;

    F8Walk cons;
    cons.b = s_b;
    cons.np = f8_seq_pages(a, s_b);
    {
        const long long rel = u0 - s_base;
        cons.j = (int)(rel / cons.np);
        cons.p = (int)(rel - (long long)cons.j * cons.np);
    }
    cons.left = u1 - u0;
    F8Walk prod = cons;

    // ---- producer: this warp's steps, segment after segment
    F8Seg ps = f8_next(a, prod, nj);
    int pst = warp, plen = min(__ldg(a.lens + ps.b), a.max_blocks * 16);
    int ids = -1, ids_at = -1;  // block ids of 32 / PP steps from step ids_at (stride W) on
    auto produce = [&](int stage) {
        // move on to a segment that has a step for this warp
        while (pst * PP >= ps.p1 - ps.p0) {
            if (prod.left <= 0) return;
            ps = f8_next(a, prod, nj);
            pst = warp;
            plen = min(__ldg(a.lens + ps.b), a.max_blocks * 16);
            ids_at = -1;
        }
        if (ids_at < 0 || pst >= ids_at + W * (32 / PP)) {
            ids_at = pst;
            const int p = ps.p0 + (pst + W * (lane / PP)) * PP + lane % PP;
            ids = p < ps.p1 ? __ldg(a.table + (int64_t)ps.b * a.max_blocks + p) : -1;
            if (p < ps.p1 && (ids < 0 || ids >= a.num_blocks)) {
                set_error(a.err, TQ_DEVERR_BLOCK);
                ids = -1;
            }
        }
        const int h = ps.j / a.nhg;
#pragma unroll
        for (int pp = 0; pp < PP; ++pp) {
            const int blk = __shfl_sync(0xffffffffu, ids, (pst - ids_at) / W * PP + pp);
            const int p = ps.p0 + pst * PP + pp;
            if (lane == 0) info[stage * PP + pp] = blk < 0 ? 0 : min(16, plen - 16 * p);
            if (blk < 0) continue;
            const uint8_t* src = a.cache + ((int64_t)blk * a.heads + h) * C::PAGE;
            const uint32_t dst = smem_u32(ring + stage * C::STEP + pp * C::PAGE);
            constexpr int CPR = D / 16;
#pragma unroll
            for (int i = 0; i < CPR; ++i) {
                // 32 rows (16 keys, 16 values) of CPR 16-byte chunks; chunk ch of
                // row r goes to ch ^ 4 (r & 1) for keys and ch ^ (r & 6) for values,
                // which the operand reads below hit without bank conflicts
                const int idx = lane + 32 * i, r = idx / CPR, ch = idx % CPR;
                const int x = r < 16 ? (r & 1) << 2 : r & 6;
                cp_async16(dst + r * D + ((ch ^ x) << 4), src + idx * 16);
            }
            if (lane < 2) cp_async16(dst + 32 * D + 16 * lane, src + 32 * D + 16 * lane);
        }
        pst += W;
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
        produce(s);
        commit();
    }
    int stage = 0;

    while (cons.left > 0) {
        const F8Seg sg = f8_next(a, cons, nj);
        const int kvh = sg.j / a.nhg, hg = sg.j - kvh * a.nhg;
        const int nh = min(a.hp, a.group - hg * a.hp);      // heads of this unit
        const int qh0 = kvh * a.group + hg * a.hp;

        // ---- query operands: fp16 of q * 2^-x with the largest in [2^8, 2^9)
        // (exact for bf16 and fp16 inputs), in fragment order
        for (int h = warp; h < HEADS; h += W) {
            float4 x[D / 128];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 128; ++i) {
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (h < nh) {
                    const int64_t off = (int64_t)sg.b * a.q_stride + (int64_t)(qh0 + h) * D + 128 * i + 4 * lane;
                    x[i] = f8_load4(static_cast<const uint8_t*>(a.q) + off * (a.q_dtype == TQ_DTYPE_F32 ? 4 : 2),
                                    a.q_dtype);
                }
                top = max(max(top, max(__float_as_uint(x[i].x) & 0x7FFFFFFFu, __float_as_uint(x[i].y) & 0x7FFFFFFFu)),
                          max(__float_as_uint(x[i].z) & 0x7FFFFFFFu, __float_as_uint(x[i].w) & 0x7FFFFFFFu));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const bool bad = top >= 0x7F800000u;
            const uint32_t e = max(top >> 23, 16u);
            const float mul = bad ? 0.f : __uint_as_float((262u - min(e, 254u)) << 23);
            if (lane == 0) cq[h] = bad ? __uint_as_float(0x7FC00000u) : a.scale_log2e * __uint_as_float((e - 8u) << 23);
#pragma unroll
            for (int i = 0; i < D / 128; ++i) {
                if (bad) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                x[i].x *= mul, x[i].y *= mul, x[i].z *= mul, x[i].w *= mul;
                // elements 128 i + 4 lane ..: 64-element half, 16-element lane part, K step
                const int el = 128 * i + 4 * lane, ks = (el >> 6) * 4 + ((el >> 2) & 3), cc = (el >> 4) & 3;
                uint2 f = make_uint2(f8_pack_f16(x[i].x, x[i].y), f8_pack_f16(x[i].z, x[i].w));
                const int at = (ks * NT + (h >> 3)) * 32 + (h & 7) * 4 + cc;
                qf[at] = f;
                if constexpr (PREC)
                    qf[(D / 16) * NT * 32 + at] =
                        make_uint2(f8_pack_rest(x[i].x, x[i].y, f.x), f8_pack_rest(x[i].z, x[i].w, f.y));
            }
        }
        __syncthreads();
        float cqr[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) cqr[n][0] = cq[8 * n + 2 * c], cqr[n][1] = cq[8 * n + 2 * c + 1];

        float o[D / 16][NT][4];
        float r[NT][2], rv[NT][2], l[NT][2];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) r[n][e] = rv[n][e] = -INFINITY, l[n][e] = 0.f;

        const int nst = (sg.p1 - sg.p0 + PP - 1) / PP;
        for (int st = warp; st < nst; st += W) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            __syncwarp();
            produce(stage == 0 ? S - 1 : stage - 1);
            commit();
            const uint8_t* sp = ring + stage * C::STEP;

            // ---- scores
            float s[PP][NT][4];
#pragma unroll
            for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                for (int n = 0; n < NT; ++n) s[pp][n][0] = s[pp][n][1] = s[pp][n][2] = s[pp][n][3] = 0.f;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                uint4 ka[PP][2];
#pragma unroll
                for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        ka[pp][u] = *reinterpret_cast<const uint4*>(sp + pp * C::PAGE + (g + 8 * u) * D +
                                                                    (((4 * h + c) ^ ((g & 1) << 2)) << 4));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int at = ((4 * h + k) * NT + n) * 32 + lane;
                        const uint2 b = qf[at];
                        uint2 bl = make_uint2(0u, 0u);
                        if constexpr (PREC) bl = qf[(D / 16) * NT * 32 + at];
#pragma unroll
                        for (int pp = 0; pp < PP; ++pp) {
                            const uint32_t w0 = k == 0 ? ka[pp][0].x : k == 1 ? ka[pp][0].y : k == 2 ? ka[pp][0].z : ka[pp][0].w;
                            const uint32_t w1 = k == 0 ? ka[pp][1].x : k == 1 ? ka[pp][1].y : k == 2 ? ka[pp][1].z : ka[pp][1].w;
                            const uint32_t a0 = f8_to_f16x2(w0), a1 = f8_to_f16x2(w1), a2 = f8_to_f16x2_hi(w0),
                                           a3 = f8_to_f16x2_hi(w1);
                            f8_mma(s[pp][n], a0, a1, a2, a3, b);
                            if constexpr (PREC) f8_mma(s[pp][n], a0, a1, a2, a3, bl);
                        }
                    }
                }
            }

            // ---- scaled scores, references
            float ev[PP][2];
            bool ok[PP][2];
            int nv[PP];
            bool moved = false;
#pragma unroll
            for (int pp = 0; pp < PP; ++pp) {
                nv[pp] = st * PP + pp < sg.p1 - sg.p0 ? info[stage * PP + pp] : 0;
                const uint8_t* ex = sp + pp * C::PAGE + 32 * D;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float ks = f8_scale(ex[g + 8 * u]);
                    const uint32_t eb = ex[16 + g + 8 * u];
                    ev[pp][u] = eb == 255u ? __uint_as_float(0x7FC00000u) : (float)((int)eb - 127);
                    ok[pp][u] = g + 8 * u < nv[pp];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& x = s[pp][n][2 * u + e];
                            x = ok[pp][u] ? x * cqr[n][e] * ks : -INFINITY;
                            moved |= x > r[n][e] + kF8Slack || x + ev[pp][u] > rv[n][e] + kF8Slack;
                        }
                }
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = -INFINITY, mv = -INFINITY;
#pragma unroll
                        for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                m = fmaxf(m, s[pp][n][2 * u + e]);
                                mv = fmaxf(mv, ok[pp][u] ? s[pp][n][2 * u + e] + ev[pp][u] : -INFINITY);
                            }
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) {
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, x));
                        }
                        m = fmaxf(r[n][e], m);
                        mv = fmaxf(rv[n][e], mv - kF8Head);
                        const float f = r[n][e] == -INFINITY ? 0.f : f8_exp2(r[n][e] - m);
                        const float fv = rv[n][e] == -INFINITY ? 0.f : f8_exp2(rv[n][e] - mv);
                        r[n][e] = m;
                        rv[n][e] = mv;
                        l[n][e] *= f;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) o[i][n][e] *= fv, o[i][n][2 + e] *= fv;
                    }
            }

            // ---- weights, as the B operand (tokens x heads)
            uint2 pb[PP][NT], pl[PP][NT];
#pragma unroll
            for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float w[4];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = s[pp][n][2 * u + e];
                            l[n][e] += ok[pp][u] ? f8_exp2(x - r[n][e]) : 0.f;
                            w[2 * u + e] = ok[pp][u] ? f8_exp2(x + ev[pp][u] - rv[n][e]) : 0.f;
                        }
                    const uint32_t h0 = f8_pack_f16(w[0], w[1]), h1 = f8_pack_f16(w[2], w[3]);
                    pb[pp][n] = make_uint2(f8_transpose(h0), f8_transpose(h1));
                    if constexpr (PREC)
                        pl[pp][n] = make_uint2(f8_transpose(f8_pack_rest(w[0], w[1], h0)),
                                               f8_transpose(f8_pack_rest(w[2], w[3], h1)));
                }

            // ---- values: token pairs (2c, 2c + 1) and (2c + 8, 2c + 9) of 16 coordinates
#pragma unroll
            for (int pp = 0; pp < PP; ++pp) {
                if (nv[pp] == 0) continue;
#pragma unroll
                for (int h = 0; h < D / 128; ++h) {
                    uint4 v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int t = 2 * c + (u & 1) + 8 * (u >> 1);
                        v[u] = *reinterpret_cast<const uint4*>(sp + pp * C::PAGE + 16 * D + t * D +
                                                               (((8 * h + g) ^ (t & 6)) << 4));
                        // rows behind the last token may hold anything
                        if (nv[pp] < 16 && t >= nv[pp]) v[u] = make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t t0 = k == 0 ? v[0].x : k == 1 ? v[0].y : k == 2 ? v[0].z : v[0].w;
                        const uint32_t t1 = k == 0 ? v[1].x : k == 1 ? v[1].y : k == 2 ? v[1].z : v[1].w;
                        const uint32_t t2 = k == 0 ? v[2].x : k == 1 ? v[2].y : k == 2 ? v[2].z : v[2].w;
                        const uint32_t t3 = k == 0 ? v[3].x : k == 1 ? v[3].y : k == 2 ? v[3].z : v[3].w;
                        const uint32_t x0 = __byte_perm(t0, t1, 0x5140), x1 = __byte_perm(t0, t1, 0x7362);
                        const uint32_t y0 = __byte_perm(t2, t3, 0x5140), y1 = __byte_perm(t2, t3, 0x7362);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t x = m ? x1 : x0, y = m ? y1 : y0;
                            const uint32_t a0 = f8_to_f16x2(x), a1 = f8_to_f16x2_hi(x), a2 = f8_to_f16x2(y),
                                           a3 = f8_to_f16x2_hi(y);
                            const int i = 8 * h + 2 * k + m;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                f8_mma(o[i][n], a0, a1, a2, a3, pb[pp][n]);
                                if constexpr (PREC) f8_mma(o[i][n], a0, a1, a2, a3, pl[pp][n]);
                            }
                        }
                    }
                }
            }
            stage = stage == S - 1 ? 0 : stage + 1;
        }

        // ---- the warps' sums become the block's, in warp order
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
                if (g == 0) {
                    float* p = ref + (warp * HEADS + 8 * n + 2 * c + e) * 3;
                    p[0] = r[n][e];
                    p[1] = rv[n][e];
                    p[2] = l[n][e];
                }
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < W; ++w) m = fmaxf(m, ref[(w * HEADS + 8 * n + 2 * c + e) * 3 + 1]);
                const float f = rv[n][e] == -INFINITY ? (l[n][e] == 0.f ? 0.f : 1.f) : f8_exp2(rv[n][e] - m);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) o[i][n][e] *= f, o[i][n][2 + e] *= f;
            }
        for (int w = 0; w < W; ++w) {
            if (warp == w) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float* p = buf + (8 * n + 2 * c + e) * C::BUF_LD + 2 * g;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            float2 x = make_float2(o[i][n][e], o[i][n][2 + e]);
                            float2* at = reinterpret_cast<float2*>(p + 16 * i);
                            if (w > 0) x.x += at->x, x.y += at->y;
                            *at = x;
                        }
                    }
            }
            __syncthreads();
        }
        // buffer position of coordinate x of a 128-wide half: 16 (x / 2 % 8) + 2 (x / 16) + x % 2
        auto pos = [](int x) { return (x & ~127) + ((x >> 1) & 7) * 16 + ((x >> 4) & 7) * 2 + (x & 1); };
        auto head_sum = [&](int h, float& R, float& Rv, float& L) {
            R = Rv = -INFINITY;
            L = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                R = fmaxf(R, ref[(w * HEADS + h) * 3]);
                Rv = fmaxf(Rv, ref[(w * HEADS + h) * 3 + 1]);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float* p = ref + (w * HEADS + h) * 3;
                L += p[0] == -INFINITY ? p[2] : p[2] * f8_exp2(p[0] - R);
            }
        };
        // 2^(r' - r) / l; no token: 0.  (A NaN sum keeps r at -inf: NaN.)
        auto norm = [](float R, float Rv, float L) {
            return L == 0.f ? 0.f : (R == -INFINITY || Rv == -INFINITY ? 1.f : exp2f(Rv - R)) / L;
        };
        const bool whole = sg.p0 == 0 && sg.p1 == sg.np;
        if (whole) {
            for (int i = tid; i < nh * (D / 2); i += kF8Threads) {
                const int h = i / (D / 2), x = 2 * (i - h * (D / 2));
                float R, Rv, L;
                head_sum(h, R, Rv, L);
                const float f = norm(R, Rv, L);
                const float2 v = *reinterpret_cast<const float2*>(buf + h * C::BUF_LD + pos(x));
                f8_store2(a.out, ((int64_t)sg.b * a.q_heads + qh0 + h) * D + x, L == 0.f ? 0.f : v.x * f,
                          L == 0.f ? 0.f : v.y * f, a.out_dtype);
            }
        } else {
            // ---- a part: to the workspace; the last block of the unit joins
            // the unit [v0, v1) of pages this segment belongs to, in run order
            const long long here = u1 - u0 - cons.left - (sg.p1 - sg.p0);  // pages of this run before the segment
            const long long v0 = u0 + here - sg.p0, v1 = v0 + sg.np;
            const long long i0 = ((v0 + 1) * N - 1) / total, i1 = (v1 * N - 1) / total;
            const int slot = blockIdx.x * 2 + (u0 >= v0 ? 0 : 1);
            float* part = a.part + (int64_t)slot * HEADS * D;
            float* meta = a.meta + (int64_t)slot * HEADS * 4;
            for (int i = tid; i < nh * D; i += kF8Threads) {
                const int h = i / D, x = i - h * D;
                part[i] = buf[h * C::BUF_LD + x];  // buffer order
            }
            if (tid < nh) {
                float R, Rv, L;
                head_sum(tid, R, Rv, L);
                meta[4 * tid] = R;
                meta[4 * tid + 1] = Rv;
                meta[4 * tid + 2] = L;
            }
            __threadfence();
            __syncthreads();
            uint32_t* cnt = a.cnt + (int64_t)sg.b * nj + sg.j;
            if (tid == 0) {
                const uint32_t old = atomicAdd(cnt, 1u);
                s_last = old == (uint32_t)(i1 - i0);
                if (s_last) *cnt = 0;  // ready for the next call
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                auto slot_of = [&](long long i) { return (int)i * 2 + (i * total / N >= v0 ? 0 : 1); };
                for (int i = tid; i < nh * (D / 2); i += kF8Threads) {
                    const int h = i / (D / 2), x = 2 * (i - h * (D / 2));
                    float R = -INFINITY, Rv = -INFINITY;
                    for (long long k = i0; k <= i1; ++k) {
                        const float* m = a.meta + ((int64_t)slot_of(k) * HEADS + h) * 4;
                        R = fmaxf(R, __ldcg(m));
                        Rv = fmaxf(Rv, __ldcg(m + 1));
                    }
                    float L = 0.f, v0f = 0.f, v1f = 0.f;
                    for (long long k = i0; k <= i1; ++k) {
                        const int64_t sl = slot_of(k);
                        const float* m = a.meta + (sl * HEADS + h) * 4;
                        const float mr = __ldcg(m), mv = __ldcg(m + 1), ml = __ldcg(m + 2);
                        const float2 v = __ldcg(reinterpret_cast<const float2*>(a.part + (sl * HEADS + h) * D + pos(x)));
                        L += mr == -INFINITY ? ml : ml * f8_exp2(mr - R);
                        const float f = mv == -INFINITY ? 1.f : f8_exp2(mv - Rv);
                        v0f += v.x * f;
                        v1f += v.y * f;
                    }
                    const float f = norm(R, Rv, L);
                    f8_store2(a.out, ((int64_t)sg.b * a.q_heads + qh0 + h) * D + x, L == 0.f ? 0.f : v0f * f,
                              L == 0.f ? 0.f : v1f * f, a.out_dtype);
                }
            }
        }
        __syncthreads();  // query operands, buffer and references are free
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int D, int NT, bool PREC>
static tq_status launch_f8_decode(const F8DecodeArgs& a, cudaStream_t s) {
    using C = F8Cfg<D, NT, PREC>;
    int sms = 0;
    tq_status st = device_sms(&sms);
    if (st != TQ_OK) return st;
    st = ensure_dynamic_smem((const void*)f8_decode_kernel<D, NT, PREC>, C::total, "f8_decode_kernel");
    if (st != TQ_OK) return st;
    // one wave of resident blocks
    const int grid = std::min(C::CTAS * sms, kF8MaxCtas);
    f8_decode_kernel<D, NT, PREC><<<grid, kF8Threads, C::total, s>>>(a);
    return cuda_status(cudaGetLastError());
}

template <int D>
static tq_status dispatch_f8_decode(const F8DecodeArgs& a, int nt, bool prec, cudaStream_t s) {
    if (nt == 1) return prec ? launch_f8_decode<D, 1, true>(a, s) : launch_f8_decode<D, 1, false>(a, s);
    return prec ? launch_f8_decode<D, 2, true>(a, s) : launch_f8_decode<D, 2, false>(a, s);
}

}  // namespace tq

using namespace tq;

extern "C" tq_status tq_f8_decode_attention(const tq_f8_cache* c, const void* q, int q_dtype, int64_t q_stride,
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
    F8DecodeArgs a;
    a.q = q;
    a.q_stride = q_stride;
    a.cache = static_cast<const uint8_t*>(cache_buf);
    a.table = block_table;
    a.lens = seq_lens;
    a.out = out;
    a.err = c->err;
    a.cnt = c->cnt;
    a.part = c->part;
    a.meta = c->meta;
    a.num_blocks = c->cfg.num_blocks;
    a.scale_log2e = (scale > 0.f ? scale : 1.0f / sqrtf((float)d)) * 1.4426950408889634f;
    a.q_dtype = q_dtype;
    a.out_dtype = out_dtype;
    a.batch = batch;
    a.heads = c->cfg.num_kv_heads;
    a.q_heads = c->cfg.num_q_heads;
    a.group = c->geom.group;
    a.nhg = c->geom.nhg;
    a.hp = c->geom.hp;
    a.max_blocks = c->cfg.max_blocks_per_seq;
    const bool prec = q_dtype == TQ_DTYPE_F32 || out_dtype == TQ_DTYPE_F32;
    cudaStream_t s = (cudaStream_t)stream;
    return d == 128 ? dispatch_f8_decode<128>(a, c->geom.nt, prec, s) : dispatch_f8_decode<256>(a, c->geom.nt, prec, s);
}
