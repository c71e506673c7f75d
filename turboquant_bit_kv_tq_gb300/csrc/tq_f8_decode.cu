// Decode attention over the 8-bit cache.
//
// With k8, v8 the codes, 2^ek, 2^ev the vectors' scales and c = scale * log2(e):
//   s_t = c <q, k8_t> 2^ek_t                    (log2 units)
//   l   = sum_t 2^(s_t - r)                     r, r + x: references of the sums, moved
//   o   = sum_t 2^((s_t - r) + (ev_t - x)) v8_t  when a weight passes 2^12
//   out = o / l * 2^x
// The value scale goes into the exponent of the weight, with a reference of its
// own, so no weight over- or underflows whatever the scales are.  That one is held
// by its distance x from r: both sums see the same difference s_t - r, exact near r
// however large the scores are, and ev_t - x keeps every digit beside it.
//
// Bound by memory (2 d + 2 bytes per token and KV head).  All pages of all
// sequences, in the order (sequence, KV head, page), are dealt out in runs to a
// fixed grid of resident blocks: evenly, one run per block, whose warps share its
// segments (the pages of one (sequence, KV head) each) step by step and add up in
// shared memory at a segment's end; or, with many short sequences, whole (sequence,
// KV head)s to warps, and no warp waits for another.  A step is 256/d pages.  Each warp
// keeps a ring of steps in flight, across segments: one tensor copy per page,
// whose 128-byte swizzle lays the rows out so that the operand reads below meet no
// bank conflict, and one small copy of its scales.  (16-byte cp.async in a swizzle
// of our own moved as much, but issuing it took a warp 1255 cycles of the 4240 of
// a step.)  Products per 16 tokens:
//   S^T[tokens x heads] = K Q^T     mma.m16n8k16, A = codes as fp16 (exact)
//   O^T[d x heads] += V^T P^T       A = pairs of value codes, B = the weights
// so a KV head's query heads (8 or 16 columns) share every page, and tokens and
// coordinates fill the 16 rows: a group of 8 heads wastes nothing.  (tcgen05
// would want 128 rows of operands in shared memory, written back after the
// conversion; mma.sync takes the converted codes from registers.)
// A segment that is a whole (sequence, KV head) is written out at once.  The
// sums of the others go to the workspace and are joined in run order by the last
// block to arrive, in groups first where there are many.
//
// Measured: 16 x 8192 tokens, 32/8 heads, d = 128: 55 us, 4.9 TB/s; 4 x up to 131072,
// 64/8 heads: 121 us, 5.6 TB/s; 8 x up to 32768, 32/4 heads, d = 256, fp32: 58 us,
// 5.1 TB/s (a plain copy: 6.8).  Longer caches add bytes at 6.3 to 6.7 TB/s; the rest
// is about 15 us a call: the first pages are under way after 3 us; of 16 x 8192, blocks
// with equal runs end between 35 and 47 us (four fifths of them between 39 and 45),
// arriving takes 1.5 and the last join up to 5.

#include <algorithm>

#include "tq_f8.cuh"
#include "tq_tma.h"

namespace tq {

struct F8DecodeArgs {
    const void* q;
    int64_t q_stride;
    const uint8_t* cache;
    const int32_t *table, *lens;
    void* out;
    uint32_t *err, *cnt, *gcnt;
    float4 *part, *meta;
    int64_t num_blocks;
    float scale_log2e;
    int q_dtype, out_dtype;
    int batch, heads, q_heads, group, nhg, hp, max_blocks;
};

constexpr int kF8Threads = 32 * kF8Warps;
// weights are kept below kF8Most and the reference is set so that the largest
// is 2^kF8Head: small weights stay normal fp16 numbers further down
constexpr float kF8Most = 4096.f, kF8Head = 4.f;
// the reference of an empty sum: no finite score lies below it, and any other is so
// far above (a unit of the last place is 2^104) that its weight moves the reference
constexpr float kF8None = -3.4028234664e38f;

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
// a page's 32 code rows: box {128 bytes, 32 rows, d/128 halves, 1 page}
__device__ __forceinline__ void f8_page_copy(uint32_t dst, const CUtensorMap* m, int page, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(dst),
        "l"(m), "r"(0), "r"(page), "r"(bar)
        : "memory");
}
// Token of row g (and, 8 further, of row g + 8) of the score product.  The swizzle
// puts 16-byte chunk x of row t at x ^ (t & 7); with this order the rows a quarter
// warp reads together differ in bit 2 (keys: rows 2i, 2i + 1, chunks c) and in
// bits 1..2 (values: rows 2c, chunks g), so that its 8 lanes hit 8 chunk places.
__device__ __forceinline__ int f8_token(int g) { return (g & 6) ^ ((g & 1) ? 5 : 0); }

template <int D, int NT, bool PREC>
struct F8Cfg {
    static constexpr int PP = 256 / D;                 // pages per step
    static constexpr int CODES = 32 * D;               // bytes of a page's codes in the ring
    static constexpr int STEP = PP * CODES;            // bytes of a ring stage
    static constexpr int HEADS = 8 * NT;
    static constexpr int QF = (D / 16) * NT * 32 * 8 * (PREC ? 2 : 1);  // query operands of a warp
    // blocks per SM (three where two stages per warp and the registers allow it,
    // else two), and as deep a ring as fits then
    static constexpr int EXTRA = PP * (32 + 4) + 8;    // scales, valid tokens and barrier of a stage
    static constexpr int per_cta(int n) { return 233472 / n - 1024 - 1280 - 1024; }
    static constexpr int fit(int n) { return (per_cta(n) / kF8Warps - QF) / (STEP + EXTRA); }
    static constexpr int CTAS = fit(3) >= 2 && NT == 1 && D == 128 ? 3 : fit(2) >= 2 ? 2 : 1;
    static constexpr int STAGES = fit(CTAS) < 6 ? fit(CTAS) : 6;
    static_assert(STAGES >= 2, "ring");
    static constexpr int off_q = kF8Warps * STAGES * STEP;
    static constexpr int off_ex = off_q + kF8Warps * QF;                   // [warps][STAGES][PP][32]
    static constexpr int off_bar = off_ex + kF8Warps * STAGES * PP * 32;   // [warps][STAGES]
    static constexpr int off_info = off_bar + kF8Warps * STAGES * 8;       // [warps][STAGES][PP] valid tokens
    static constexpr int total = off_info + kF8Warps * STAGES * PP * 4 + 1024;  // + alignment to 1024
    static constexpr int ITEMS = D / 16 * NT * 32;     // float4 per partial sum
    // the join's factors, then partial sums, in place of rings and query operands
    static constexpr int JOIN_AT = 4096;
    static constexpr int JOIN_FIT = (off_ex - JOIN_AT) / (ITEMS * 16), JOIN_CAP = JOIN_FIT < 32 ? JOIN_FIT : 32;
    static_assert(JOIN_CAP >= 1, "place for a join");
    // two sums fit the four warps' query operands, whose place they take at a segment's end
    static_assert(2 * ITEMS * 16 <= kF8Warps * QF, "merge buffers");
};
static_assert(kF8Ctas >= F8Cfg<128, 1, false>::CTAS, "workspace slots");

__device__ __forceinline__ int f8_clamp(const F8DecodeArgs& a, int len) { return max(0, min(len, a.max_blocks * 16)); }
__device__ __forceinline__ int f8_pages(const F8DecodeArgs& a, int len) { return (f8_clamp(a, len) + 15) >> 4; }

// A unit (a sequence's KV head and head group) costs more than its pages (its query,
// its sums): in the order that is dealt out `cost` empty places follow its last.
__device__ __forceinline__ int f8_places(int np, int cost) { return np > 0 ? np + cost : 0; }

// A position in the order (sequence, KV head and head group, page) and the
// places left of a run.
struct F8Walk {
    int b, j, p, len, left, at;
};
struct F8Seg {
    int b, j, p0, p1, len, v0;  // pages [p0, p1), none if the run has only empty places of the unit; v0: place of page 0
    __device__ __forceinline__ int np() const { return (len + 15) >> 4; }
};
__device__ __forceinline__ F8Seg f8_next(const F8DecodeArgs& a, F8Walk& w, int nj, int cost) {
    F8Seg s;
    s.b = w.b;
    s.j = w.j;
    s.len = w.len;
    s.v0 = w.at - w.p;
    const int np = s.np(), n = min(f8_places(np, cost) - w.p, w.left);
    s.p0 = min(w.p, np);
    s.p1 = min(w.p + n, np);
    w.left -= n;
    w.at += n;
    w.p = 0;
    if (++w.j == nj) {
        w.j = 0;
        w.len = 0;
        while (w.left > 0 && w.len == 0 && ++w.b < a.batch) w.len = f8_clamp(a, __ldg(a.lens + w.b));
    }
    return s;
}

// Even runs: run i < n takes units [start(i), start(i + 1)) of `total` >= n.
struct F8Runs {
    uint32_t q, r, n;
    __device__ __forceinline__ uint32_t start(uint32_t i) const { return i * q + min(i, r); }
    __device__ __forceinline__ uint32_t owner(uint32_t u) const {
        const uint32_t big = r * (q + 1);
        return u < big ? u / (q + 1) : r + (u - big) / q;
    }
};

// 2^x / l of a head's sums, as two factors: the power alone is subnormal where the
// value scales are the smallest.  No token: 0
__device__ __forceinline__ float2 f8_norm(float X, float L) {
    const float half = exp2f(0.5f * X);
    return L == 0.f ? make_float2(0.f, 0.f) : make_float2(half / L, half);
}

constexpr int kF8SoloPages = 16;  // a warp takes units of up to this many pages alone, whatever its share
// The parts of up to kF8Join blocks are joined by the last of them; of more, by the
// last of each kF8Group, and the groups' by the last group (one KV head, 32768 tokens
// = 128 blocks: 21 us in groups of 16, 25 in groups of 32; 8 x up to 32768 with at most
// 18 blocks a unit: 70 us in one step).
constexpr int kF8Join = 32, kF8Group = 16;
struct F8JoinSmem {
    float fac[kF8Join][16];
    float4 tot[16];  // {r, x, l, -} for another join, {f8_norm's factors, l, -} for the output
};
static_assert(kF8Join <= 32 && kF8MaxSms * kF8Ctas / kF8Group + 1 <= kF8Join, "groups of a join");

template <int D, int NT, bool PREC>
__global__ void __launch_bounds__(kF8Threads, F8Cfg<D, NT, PREC>::CTAS) f8_decode_kernel(const __grid_constant__ F8DecodeArgs a, const __grid_constant__ CUtensorMap pages) {
    using C = F8Cfg<D, NT, PREC>;
    constexpr int S = C::STAGES, PP = C::PP, W = kF8Warps, HEADS = C::HEADS;
    static_assert(sizeof(F8JoinSmem) <= C::JOIN_AT, "the join reuses the rings");
    extern __shared__ uint8_t raw[];
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    __shared__ int s_last[2][2];  // [unit][level]: each written once, so that no read of one is overtaken
    __shared__ float4 s_ref[W][HEADS];
    __shared__ uint64_t s_jbar;  // the joins' copies
    __shared__ F8Seg s_part[2];  // segments whose sums are in the workspace (b < 0: none)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int nj = a.heads * a.nhg;
    uint8_t* ring = smem + warp * (S * C::STEP);
    uint2* qf = reinterpret_cast<uint2*>(smem + C::off_q + warp * C::QF);
    const uint8_t* exps = smem + C::off_ex + warp * S * PP * 32;
    const uint32_t bars = smem_u32(smem + C::off_bar) + warp * S * 8;
    int* info = reinterpret_cast<int*>(smem + C::off_info) + warp * S * PP;
    const int tok = f8_token(g);
    bool dead = false;
    const uint32_t jbar = smem_u32(&s_jbar);
    if (tid == 0) mbar_init(jbar, 1);
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();

    if (tid < 2) s_part[tid].b = -1;  // (warp 0 alone writes them, and all read after a barrier)
    pdl_wait();
    // ---- totals: lane i of every warp counts the sequences [i per, (i + 1) per)
    const int per = (a.batch + 31) >> 5;
    const int bt0 = min(a.batch, lane * per), bt1 = min(a.batch, bt0 + per);
    int mine = 0, some = 0, most = 0;
#pragma unroll 4
    for (int b = bt0; b < bt1; ++b) {
        const int len = __ldg(a.lens + b);
        if (len < 0 || len > a.max_blocks * 16) set_error(a.err, TQ_DEVERR_SEQLEN);
        const int np = f8_pages(a, len);
        mine += np;
        some += np > 0;
        most = max(most, np);
    }
    const int units = (int)__reduce_add_sync(0xffffffffu, (unsigned)some) * nj;
    const int all_pages = (int)__reduce_add_sync(0xffffffffu, (unsigned)mine) * nj;
    most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
    // One run per block, of at least 16 pages on average (two steps for each
    // warp); or, with more units than blocks and none much longer than a warp's
    // share, a run of whole units per warp (256 x 100 tokens, 8 KV heads: 22 us, block
    // runs 30; 256 x up to 200: 21, 37; 512 x up to 400: 53, 69).
    const int warps = (int)gridDim.x * W, share = all_pages / warps;
    const bool solo = units > (int)gridDim.x && most <= max(kF8SoloPages, 2 * share);
    // (a fixed cost, of less weight where the runs are short: the last of several runs
    // of a unit would be left with few pages)
    const int cost = min(kF8UnitCost, share);
    mine += cost * some;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    const int before = (incl - mine) * nj, total = all_pages + cost * units;
    // sequences without a token: their rows are zero
    if (units < a.batch * nj)
        for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
            if (f8_pages(a, __ldg(a.lens + b)) > 0) continue;
            for (int i = tid; i < a.q_heads * D / 2; i += kF8Threads)
                f8_store2(a.out, (int64_t)b * a.q_heads * D + 2 * i, 0.f, 0.f, a.out_dtype);
        }
    if (total == 0) return;
    F8Runs runs;
    runs.n = solo ? (uint32_t)min(warps, total)
                  : (uint32_t)min((long long)gridDim.x, (long long)units * max(1, all_pages / units / 16));
    runs.q = (uint32_t)total / runs.n;
    runs.r = (uint32_t)total - runs.q * runs.n;
    const uint32_t run = solo ? blockIdx.x * W + warp : blockIdx.x;

    if (run < runs.n) {
        const int sw = solo ? 0 : warp, sn = solo ? 1 : W;  // this warp takes the steps sw, sw + sn, ... of a segment
        // page u of the order: one lane has its sequence among its own
        auto locate = [&](int u) {
            int at = before, b = bt0, len = 0;
            const bool here = u >= before && u < before + mine * nj;
            if (here)
                for (;; ++b) {
                    len = __ldg(a.lens + b);
                    const int n = f8_places(f8_pages(a, len), cost) * nj;
                    if (u < at + n) break;
                    at += n;
                }
            const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
            F8Walk w;
            w.b = __shfl_sync(0xffffffffu, b, src);
            w.len = f8_clamp(a, __shfl_sync(0xffffffffu, len, src));
            const int rel = u - __shfl_sync(0xffffffffu, at, src), np = f8_places((w.len + 15) >> 4, cost);
            w.j = rel / np;
            w.p = rel - w.j * np;
            w.left = total - u;
            w.at = u;
            return w;
        };
        int u0 = (int)runs.start(run), u1 = (int)runs.start(run + 1);
        F8Walk cons = locate(u0);
        if (solo) {
            // the units that start in [u0, u1)
            if (u1 < total) {
                const F8Walk w = locate(u1);
                if (w.p > 0) u1 += f8_places((w.len + 15) >> 4, cost) - w.p;
            }
            if (cons.p > 0) {
                u0 += f8_places((cons.len + 15) >> 4, cost) - cons.p;
                f8_next(a, cons, nj, cost);
            }
        }
        cons.left = u1 - u0;
        if (cons.left <= 0) return;  // (solo: no unit starts here)
        F8Walk prod = cons;

        // ---- producer: this warp's steps, segment after segment
        F8Seg ps = f8_next(a, prod, nj, cost);
        int pst = sw;
        int made = 0, used = 0;  // steps copied, steps taken
        int ids = -1, ids_at = 0, ids_n = 0;  // block ids of ids_n pages: this warp's steps from ids_at on
        auto produce = [&](int stage) {
            while (ps.p0 + pst * PP >= ps.p1) {
                if (prod.left <= 0) return;
                ps = f8_next(a, prod, nj, cost);
                pst = sw;
                ids_n = 0;
            }
            if (ids_at >= ids_n) {
                ids_at = 0;
                ids_n = 32;
                const int p = ps.p0 + (pst + sn * (lane / PP)) * PP + lane % PP;
                ids = p < ps.p1 ? __ldg(a.table + (int64_t)ps.b * a.max_blocks + p) : -1;
                if (p < ps.p1 && (ids < 0 || ids >= a.num_blocks)) {
                    set_error(a.err, TQ_DEVERR_BLOCK);
                    ids = -1;
                }
            }
            const int h = a.nhg == 1 ? ps.j : ps.j / a.nhg;
            // lane pp: page pp of the step (one behind the segment's last has block id -1 too)
            const int blk = __shfl_sync(0xffffffffu, ids, ids_at + (lane < PP ? lane : 0));
            const bool there = lane < PP && blk >= 0;
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, there));
            if (lane == 0) mbar_expect_tx(bars + 8 * stage, n * f8_page_bytes(D));
            if (lane < PP) info[stage * PP + lane] = there ? min(16, ps.len - 16 * (ps.p0 + pst * PP + lane)) : 0;
            __syncwarp();
            if (there) {
                const int page = blk * a.heads + h;
                f8_page_copy(smem_u32(ring) + stage * C::STEP + lane * C::CODES, &pages, page, bars + 8 * stage);
                bulk_copy(smem_u32(exps) + (stage * PP + lane) * 32, a.cache + (int64_t)page * f8_page_bytes(D) + C::CODES, 32,
                          bars + 8 * stage);
            }
            pst += sn;
            ids_at += PP;
            ++made;
        };
#pragma unroll
        for (int s = 0; s < S - 1; ++s) produce(s);
        int stage = 0;

        while (cons.left > 0) {
            const F8Seg sg = f8_next(a, cons, nj, cost);
            if (sg.p0 == sg.p1) continue;
            const int kvh = a.nhg == 1 ? sg.j : sg.j / a.nhg, hg = sg.j - kvh * a.nhg;
            const int nh = min(a.hp, a.group - hg * a.hp);  // heads of this unit
            const int qh0 = kvh * a.group + hg * a.hp;

            // ---- query operands: fp16 of q * 2^-x with the largest in [2^8, 2^9), in
            // fragment order.  Exact for fp16 elements down to 2^-22 of the head's largest
            // and bf16 ones down to 2^-25; below, they are rounded to steps of at most 2^-32
            // of it, which is less than the fp32 score's rounding
            float cqr[NT][2];
            constexpr int QB = HEADS * D <= 8 * 128 ? 8 : 4;  // heads loaded at once
            const int64_t qoff = (int64_t)sg.b * a.q_stride + (int64_t)qh0 * D + 4 * lane;
#pragma unroll
            for (int h8 = 0; h8 < HEADS; h8 += QB) {
                float4 x[QB][D / 128];
                if (PREC && a.q_dtype == TQ_DTYPE_F32) {
#pragma unroll
                    for (int hh = 0; hh < QB; ++hh)
#pragma unroll
                        for (int i = 0; i < D / 128; ++i)
                            x[hh][i] = h8 + hh < nh ? __ldg(reinterpret_cast<const float4*>(
                                                          static_cast<const float*>(a.q) + qoff + (h8 + hh) * D + 128 * i))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                } else {
                    uint2 y[QB][D / 128];
#pragma unroll
                    for (int hh = 0; hh < QB; ++hh)
#pragma unroll
                        for (int i = 0; i < D / 128; ++i)
                            y[hh][i] = h8 + hh < nh ? __ldg(reinterpret_cast<const uint2*>(
                                                          static_cast<const uint16_t*>(a.q) + qoff + (h8 + hh) * D + 128 * i))
                                                    : make_uint2(0u, 0u);
                    const bool bf = a.q_dtype == TQ_DTYPE_BF16;
#pragma unroll
                    for (int hh = 0; hh < QB; ++hh)
#pragma unroll
                        for (int i = 0; i < D / 128; ++i) {
                            const float2 u = bf ? F8Elem::from_bf16x2(y[hh][i].x) : F8Elem::from_f16x2(y[hh][i].x);
                            const float2 w = bf ? F8Elem::from_bf16x2(y[hh][i].y) : F8Elem::from_f16x2(y[hh][i].y);
                            x[hh][i] = make_float4(u.x, u.y, w.x, w.y);
                        }
                }
#pragma unroll
                for (int hh = 0; hh < QB; ++hh) {
                    const int h = h8 + hh;
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < D / 128; ++i)
                        top = max(max(top, max(__float_as_uint(x[hh][i].x) & 0x7FFFFFFFu,
                                               __float_as_uint(x[hh][i].y) & 0x7FFFFFFFu)),
                                  max(__float_as_uint(x[hh][i].z) & 0x7FFFFFFFu,
                                      __float_as_uint(x[hh][i].w) & 0x7FFFFFFFu));
                    top = __reduce_max_sync(0xffffffffu, top);
                    const bool bad = top >= 0x7F800000u;
                    const uint32_t e = max(top >> 23, 16u);
                    const float mul = bad ? 0.f : __uint_as_float((262u - min(e, 254u)) << 23);
                    const float cq =
                        bad ? __uint_as_float(0x7FC00000u) : a.scale_log2e * __uint_as_float((e - 8u) << 23);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            if (8 * n + 2 * c + u == h) cqr[n][u] = cq;
#pragma unroll
                    for (int i = 0; i < D / 128; ++i) {
                        float4 y = x[hh][i];
                        if (bad) y = make_float4(0.f, 0.f, 0.f, 0.f);
                        y.x *= mul, y.y *= mul, y.z *= mul, y.w *= mul;
                        // elements 128 i + 4 lane ..: 64-element half, K step, 16-element lane part
                        const int el = 128 * i + 4 * lane, ks = (el >> 6) * 4 + ((el >> 2) & 3), cc = (el >> 4) & 3;
                        const uint2 f = make_uint2(f8_pack_f16(y.x, y.y), f8_pack_f16(y.z, y.w));
                        const int at = (ks * NT + (h >> 3)) * 32 + (h & 7) * 4 + cc;
                        qf[at] = f;
                        if constexpr (PREC)
                            qf[(D / 16) * NT * 32 + at] =
                                make_uint2(f8_pack_rest(y.x, y.y, f.x), f8_pack_rest(y.z, y.w, f.y));
                    }
                }
            }

            float o[D / 16][NT][4];
            float r[NT][2], xv[NT][2], l[NT][2];
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) r[n][e] = kF8None, xv[n][e] = l[n][e] = 0.f;

            for (int p = sg.p0 + sw * PP; p < sg.p1; p += sn * PP) {
                __syncwarp();  // the last step's stage (and qf) is settled
                if (!dead) produce(stage == 0 ? S - 1 : stage - 1);
                if (!dead) dead = !mbar_wait(bars + 8 * stage, (used / S) & 1, a.err);
                dead = __any_sync(0xffffffffu, dead);
                ++used;
                const uint8_t* sp = ring + stage * C::STEP;
                // ---- scores
                // chains of dependent products: one per page and n-tile, two more where
                // that is only one, and the queries' second parts in their own
                constexpr int CH = PP * NT == 1 ? 2 : 1, ACC = CH * (PREC ? 2 : 1);
                float acc[ACC][PP][NT][4];
#pragma unroll
                for (int x = 0; x < ACC; ++x)
#pragma unroll
                    for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            acc[x][pp][n][0] = acc[x][pp][n][1] = acc[x][pp][n][2] = acc[x][pp][n][3] = 0.f;
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    uint4 ka[PP][2];
#pragma unroll
                    for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            ka[pp][u] = *reinterpret_cast<const uint4*>(
                                sp + pp * C::CODES + (h >> 1) * 4096 + (tok + 8 * u) * 128 + (((4 * (h & 1) + c) ^ tok) << 4));
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
                                f8_mma(acc[k % CH][pp][n], a0, a1, a2, a3, b);
                                if constexpr (PREC) f8_mma(acc[CH + k % CH][pp][n], a0, a1, a2, a3, bl);
                            }
                        }
                    }
                }
                float s[PP][NT][4];
#pragma unroll
                for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            s[pp][n][i] = acc[ACC - 1][pp][n][i];
#pragma unroll
                            for (int x = ACC - 2; x >= 0; --x) s[pp][n][i] += acc[x][pp][n][i];
                        }

                // ---- weights.  p = 2^(s - r), w = 2^((s - r) + (ev - x))
                float ev[PP][2], pw[PP][NT][4], w[PP][NT][4], top = 0.f;
                int nv[PP];
                bool full = true;
#pragma unroll
                for (int pp = 0; pp < PP; ++pp) {
                    nv[pp] = info[stage * PP + pp];
                    full &= nv[pp] == 16;
                    const uint8_t* ex = exps + (stage * PP + pp) * 32;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        // a vector stored as NaN has zero codes and E = 255: 0 * inf here
                        // (0 stands for 2^-127, a subnormal)
                        const float ck = __uint_as_float(max((uint32_t)ex[tok + 8 * u] << 23, 0x00400000u));
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) s[pp][n][2 * u + e] = __fmul_rn(s[pp][n][2 * u + e], ck * cqr[n][e]);
                        const uint32_t eb = ex[16 + tok + 8 * u];
                        ev[pp][u] = eb == 255u ? __uint_as_float(0x7FC00000u)
                                               : __uint_as_float(0x4B000000u | eb) - (8388608.f + 127.f);
                    }
                }
                auto weights = [&]() {
#pragma unroll
                    for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    // (a product and a difference, not one fma: the largest
                                    // score is 0 away from itself)
                                    const float x = __fsub_rn(s[pp][n][2 * u + e], r[n][e]);
                                    pw[pp][n][2 * u + e] = f8_exp2(x);
                                    w[pp][n][2 * u + e] = f8_exp2(x + (ev[pp][u] - xv[n][e]));
                                }
                    if (!full) {
#pragma unroll
                        for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (tok + 8 * (i >> 1) >= nv[pp]) pw[pp][n][i] = w[pp][n][i] = 0.f;
                    }
                };
                weights();
#pragma unroll
                for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(pw[pp][n][i], w[pp][n][i]));
                if (__any_sync(0xffffffffu, top > kF8Most)) {
                    // a weight has outgrown its reference: move the references
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = r[n][e];
#pragma unroll
                            for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                                for (int u = 0; u < 2; ++u)
                                    if (tok + 8 * u < nv[pp]) m = fmaxf(m, s[pp][n][2 * u + e]);
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            const float was = (r[n][e] - m) + xv[n][e];  // the old r + x, from m
                            float mv = was + kF8Head;
#pragma unroll
                            for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                                for (int u = 0; u < 2; ++u)
                                    if (tok + 8 * u < nv[pp]) mv = fmaxf(mv, (s[pp][n][2 * u + e] - m) + ev[pp][u]);
                            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, 4));
                            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, 8));
                            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, 16)) - kF8Head;
                            const float fv = f8_exp2(was - mv);
                            l[n][e] *= f8_exp2(r[n][e] - m);
                            r[n][e] = m;
                            xv[n][e] = mv;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) o[i][n][e] *= fv, o[i][n][2 + e] *= fv;
                        }
                    weights();
                }
                uint2 pb[PP][NT], pl[PP][NT];  // as the B operand (tokens x heads)
#pragma unroll
                for (int pp = 0; pp < PP; ++pp)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        l[n][0] += pw[pp][n][0] + pw[pp][n][2];
                        l[n][1] += pw[pp][n][1] + pw[pp][n][3];
                        const float* x = w[pp][n];
                        const uint32_t h0 = f8_pack_f16(x[0], x[1]), h1 = f8_pack_f16(x[2], x[3]);
                        pb[pp][n] = make_uint2(f8_transpose(h0), f8_transpose(h1));
                        if constexpr (PREC)
                            pl[pp][n] = make_uint2(f8_transpose(f8_pack_rest(x[0], x[1], h0)),
                                                   f8_transpose(f8_pack_rest(x[2], x[3], h1)));
                    }

                // ---- values: the token pairs of rows (2c, 2c + 1) and (2c + 8, 2c + 9), 16 coordinates
                if (!full) {
                    // rows behind the last token may hold anything, NaN codes too
#pragma unroll 1
                    for (int idx = lane; idx < PP * D; idx += 32) {
                        const int pp = idx / D, x = idx % D, t = x / 8 % 16;  // 16-byte piece x of the page's value rows
                        if (t >= info[stage * PP + pp])
                            *reinterpret_cast<uint4*>(ring + stage * C::STEP + pp * C::CODES + (x / 128) * 4096 + 2048 +
                                                      (x % 128) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the stage's next copy
                    __syncwarp();
                }
                // The tensor cores cut their sums off instead of rounding them: half a unit
                // lost with every product, always toward zero.  With fp32 in or out a step's
                // products are summed apart, smaller parts first, and added with a rounding (4
                // x up to 63851 tokens, 8 heads, d = 128: an error of 4.5e-7 instead of 3.9e-6).
                constexpr int VP = PREC ? PP : 1;  // pages whose products are summed apart
#pragma unroll
                for (int p0 = 0; p0 < PP; p0 += VP) {
                    if (VP == 1 && nv[p0] == 0) continue;
#pragma unroll
                    for (int h = 0; h < D / 128; ++h) {
                        uint4 v[VP][4];
#pragma unroll
                        for (int pp = 0; pp < VP; ++pp)
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int t = f8_token(2 * c + (u & 1));
                                v[pp][u] = *reinterpret_cast<const uint4*>(sp + (p0 + pp) * C::CODES + h * 4096 + 2048 +
                                                                           (t + 8 * (u >> 1)) * 128 + ((g ^ t) << 4));
                            }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t va[VP][2][4];
#pragma unroll
                            for (int pp = 0; pp < VP; ++pp) {
                                auto word = [&](int u) {
                                    return k == 0 ? v[pp][u].x : k == 1 ? v[pp][u].y : k == 2 ? v[pp][u].z : v[pp][u].w;
                                };
                                const uint32_t t0 = word(0), t1 = word(1), t2 = word(2), t3 = word(3);
                                const uint32_t x0 = __byte_perm(t0, t1, 0x5140), x1 = __byte_perm(t0, t1, 0x7362);
                                const uint32_t y0 = __byte_perm(t2, t3, 0x5140), y1 = __byte_perm(t2, t3, 0x7362);
#pragma unroll
                                for (int m = 0; m < 2; ++m) {
                                    const uint32_t x = m ? x1 : x0, y = m ? y1 : y0;
                                    va[pp][m][0] = f8_to_f16x2(x), va[pp][m][1] = f8_to_f16x2_hi(x);
                                    va[pp][m][2] = f8_to_f16x2(y), va[pp][m][3] = f8_to_f16x2_hi(y);
                                }
                            }
                            auto product = [&](float (&to)[4], int pp, int m, uint2 b) {
                                f8_mma(to, va[pp][m][0], va[pp][m][1], va[pp][m][2], va[pp][m][3], b);
                            };
                            if constexpr (PREC) {
#pragma unroll
                                for (int m = 0; m < 2; ++m) {
                                    float t[NT][4] = {};
#pragma unroll
                                    for (int part = 1; part >= 0; --part)
#pragma unroll
                                        for (int pp = 0; pp < VP; ++pp)
#pragma unroll
                                            for (int n = 0; n < NT; ++n)
                                                product(t[n], pp, m, part ? pl[p0 + pp][n] : pb[p0 + pp][n]);
#pragma unroll
                                    for (int n = 0; n < NT; ++n)
#pragma unroll
                                        for (int i = 0; i < 4; ++i) o[8 * h + 2 * k + m][n][i] += t[n][i];
                                }
                            } else {
#pragma unroll
                                for (int m = 0; m < 2; ++m)
#pragma unroll
                                    for (int n = 0; n < NT; ++n) product(o[8 * h + 2 * k + m][n], 0, m, pb[p0][n]);
                            }
                        }
                    }
                }
                stage = stage == S - 1 ? 0 : stage + 1;
            }

            // ---- the segment's sums
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
            if (!solo) {
                // the warps' sums, (0 + 2) + (1 + 3), in warp 0's registers
                float4* buf = reinterpret_cast<float4*>(smem + C::off_q);
                if (g == 0)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            s_ref[warp][8 * n + 2 * c + e] = make_float4(r[n][e], xv[n][e], l[n][e], 0.f);
                __syncthreads();
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float R = kF8None, X = -INFINITY, L = 0.f;
                        float4 m[W];
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            m[w] = s_ref[w][8 * n + 2 * c + e];
                            R = fmaxf(R, m[w].x);
                        }
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            X = fmaxf(X, (m[w].x - R) + m[w].y);
                            L += m[w].z * f8_exp2(m[w].x - R);
                        }
                        const float f = f8_exp2(((r[n][e] - R) + xv[n][e]) - X);
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) o[i][n][e] *= f, o[i][n][2 + e] *= f;
                        r[n][e] = R;
                        xv[n][e] = X;
                        l[n][e] = L;
                    }
                auto put = [&](int at) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            buf[at * C::ITEMS + (i * NT + n) * 32 + lane] =
                                make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
                };
                auto add = [&](int at) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float4 x = buf[at * C::ITEMS + (i * NT + n) * 32 + lane];
                            o[i][n][0] += x.x, o[i][n][1] += x.y, o[i][n][2] += x.z, o[i][n][3] += x.w;
                        }
                };
                if (warp >= 2) put(warp - 2);
                __syncthreads();
                if (warp < 2) add(warp);
                if (warp == 1) put(1);
                __syncthreads();
                if (warp == 0) add(1);
                __syncthreads();  // the query operands' place is free
            }
            if (!solo && warp != 0) {
                // warp 0 has the sums
            } else if (sg.p0 == 0 && sg.p1 == sg.np()) {
                // lane (g, c): coordinates 16 g .. 16 g + 15 of each 128, heads 2c and 2c + 1
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int h = 8 * n + 2 * c + e;
                        const float2 f = f8_norm(xv[n][e], l[n][e]);
                        if (h < nh)
#pragma unroll
                            for (int i0 = 0; i0 < D / 16; i0 += 8) {
                                float v[16];
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    v[2 * i] = l[n][e] == 0.f ? 0.f : o[i0 + i][n][e] * f.x * f.y;
                                    v[2 * i + 1] = l[n][e] == 0.f ? 0.f : o[i0 + i][n][2 + e] * f.x * f.y;
                                }
                                f8_store16(a.out, ((int64_t)sg.b * a.q_heads + qh0 + h) * D + 16 * i0 + 16 * g, v,
                                           a.out_dtype);
                            }
                    }
            } else {
                const int which = u0 >= sg.v0 ? 0 : 1;  // 0: the run starts in this unit
                const int slot = 2 * (int)run + which;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        a.part[(int64_t)slot * C::ITEMS + (i * NT + n) * 32 + lane] =
                            make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
                if (g == 0)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            a.meta[slot * HEADS + 8 * n + 2 * c + e] = make_float4(r[n][e], xv[n][e], l[n][e], 0.f);
                if (lane == 0) s_part[which] = sg;
            }
            __syncwarp();  // qf is free
        }
        // after a wait that gave up: copies still in flight land before the ring is reused
        if (dead)
            for (bool d2 = false; used < made; ++used)
                if (!d2) d2 = !mbar_wait(bars + 8 * (used % S), (used / S) & 1, a.err);
    }

    if (solo) return;

    // ---- joins
    __syncthreads();  // the rings are free, the block's sums written
    F8JoinSmem& js = *reinterpret_cast<F8JoinSmem*>(smem);
    int joined = 0;
    // the sums of `count` <= 32 slots (s0, then s1 + st, s1 + 2 st, ...) into slot s0, or out
    auto join = [&](int count, int s0, int s1, int st, bool fin, const F8Seg& sg) {
        auto slot = [&](int k) { return (int64_t)(k == 0 ? s0 : s1 + k * st); };
        constexpr int IPT = C::ITEMS / kF8Threads;
        static_assert(C::ITEMS % kF8Threads == 0, "items of a thread");
        float4 v[IPT];
#pragma unroll
        for (int y = 0; y < IPT; ++y) v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k0 = 0; k0 < count; k0 += C::JOIN_CAP) {
            const int n = min(C::JOIN_CAP, count - k0);
            // the sums come by bulk copies, all under way at once; lane k: slot k0 + k
            if (warp == 0) {
                if (lane == 0) mbar_expect_tx(jbar, n * (C::ITEMS * 16));
                __syncwarp();
                if (lane < n) {
                    // other blocks' plain writes, and this block's last use of the place, before the copy
                    asm volatile("fence.proxy.async;" ::: "memory");
                    bulk_copy(smem_u32(smem) + C::JOIN_AT + lane * (C::ITEMS * 16), a.part + slot(k0 + lane) * C::ITEMS,
                              C::ITEMS * 16, jbar);
                }
            }
            if (k0 == 0) {
                // lane k: slot k
                float4 ms[HEADS / W];
#pragma unroll
                for (int y = 0; y < HEADS / W; ++y)
                    ms[y] = lane < count ? __ldcg(a.meta + slot(lane) * HEADS + warp + y * W)
                                         : make_float4(kF8None, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < HEADS / W; ++y) {
                    const int h = warp + y * W;
                    const float4 m = ms[y];
                    const float R = warp_max(m.x), at = (m.x - R) + m.y, X = warp_max(at);
                    const float L = warp_sum(m.z * f8_exp2(m.x - R));
                    js.fac[lane][h] = f8_exp2(at - X);
                    const float2 f = f8_norm(X, L);
                    if (lane == 0) js.tot[h] = fin ? make_float4(f.x, f.y, L, 0.f) : make_float4(R, X, L, 0.f);
                }
                __syncthreads();  // the factors
            }
            if (!mbar_wait(jbar, joined & 1, a.err)) mbar_wait(jbar, joined & 1, a.err);
            ++joined;
            const float4* x = reinterpret_cast<const float4*>(smem + C::JOIN_AT) + tid;
#pragma unroll 2
            for (int k = 0; k < n; ++k) {
#pragma unroll
                for (int y = 0; y < IPT; ++y) {
                    const int it = tid + y * kF8Threads, h = 8 * ((it >> 5) % NT) + 2 * (it & 3);
                    const float4 z = x[k * C::ITEMS + y * kF8Threads];
                    const float2 f = *reinterpret_cast<const float2*>(&js.fac[k0 + k][h]);
                    v[y].x += z.x * f.x, v[y].y += z.y * f.y, v[y].z += z.z * f.x, v[y].w += z.w * f.y;
                }
            }
            __syncthreads();  // the place is free
        }
        const int kvh = sg.j / a.nhg, hg = sg.j - kvh * a.nhg;
        const int nh = min(a.hp, a.group - hg * a.hp), qh0 = kvh * a.group + hg * a.hp;
#pragma unroll
        for (int y = 0; y < IPT; ++y) {
            const int it = tid + y * kF8Threads;
            const int ln = it & 31, n = (it >> 5) % NT, i = (it >> 5) / NT, h = 8 * n + 2 * (ln & 3);
            if (!fin) {
                a.part[(int64_t)s0 * C::ITEMS + it] = v[y];
            } else if (h < nh) {
                const float4 t0 = js.tot[h], t1 = js.tot[h + 1];
                const int64_t at = ((int64_t)sg.b * a.q_heads + qh0 + h) * D + (i >> 3) * 128 + 16 * (ln >> 2) + 2 * (i & 7);
                f8_store2(a.out, at, t0.z == 0.f ? 0.f : v[y].x * t0.x * t0.y, t0.z == 0.f ? 0.f : v[y].z * t0.x * t0.y,
                          a.out_dtype);
                if (h + 1 < nh)
                    f8_store2(a.out, at + D, t1.z == 0.f ? 0.f : v[y].y * t1.x * t1.y,
                              t1.z == 0.f ? 0.f : v[y].w * t1.x * t1.y, a.out_dtype);
            }
        }
        if (!fin && tid < HEADS) a.meta[s0 * HEADS + tid] = js.tot[tid];
        __syncthreads();
    };
    // one more of `all` has arrived at *cnt, seen by one thread after a barrier: is it
    // the last?  (leaves the counter ready for the next call)
    auto arrive = [&](uint32_t* cnt, int all) {
        __threadfence();  // the block's writes
        const bool last = atomicAdd(cnt, 1u) == (uint32_t)(all - 1);
        if (last) *cnt = 0;
        __threadfence();
        return last;
    };
    // What a block's part of a unit is joined with: the runs (= blocks) of the unit,
    // c0 .. c1, from the one that holds its first page on; with more than kF8Join of
    // them in groups first.
    struct Step {
        int jn, j0, j1, st;  // sums to join: slots j0, then j1 + st, j1 + 2 st, ...
        uint32_t* cnt;
    };
    auto step = [&](const F8Seg& sg, bool fin, bool& single) {
        const int c0 = (int)runs.owner(sg.v0), c1 = (int)runs.owner(sg.v0 + sg.np() - 1), n = c1 - c0 + 1;
        const int first = 2 * c0 + ((int)runs.start(c0) >= sg.v0 ? 0 : 1);  // slot of block c0; the others': 2 c
        const int gi = ((int)run - c0) / kF8Group, g0 = c0 + gi * kF8Group;
        single = n <= kF8Join;
        Step s;
        if (single || fin) {
            s.jn = single ? n : (n + kF8Group - 1) / kF8Group;
            s.j0 = first;
            s.j1 = 2 * c0;
            s.st = single ? 2 : 2 * kF8Group;
            s.cnt = a.cnt + (int64_t)sg.b * nj + sg.j;
        } else {
            s.jn = min(kF8Group, c1 - g0 + 1);
            s.j0 = gi == 0 ? first : 2 * g0;
            s.j1 = 2 * g0;
            s.st = 2;
            s.cnt = a.gcnt + s.j0;
        }
        return s;
    };
    // a block may hold the end of one unit and the beginning of another: both arrive at once
    if (lane == 0 && warp < 2) {
        bool single;
        s_last[warp][0] = 0;
        if (s_part[warp].b >= 0) {
            const Step s = step(s_part[warp], false, single);
            s_last[warp][0] = arrive(s.cnt, s.jn);
        }
    }
    __syncthreads();
    for (int x = 0; x < 2; ++x) {
        if (!s_last[x][0]) continue;
        const F8Seg sg = s_part[x];
        bool single;
        Step s = step(sg, false, single);
        if (s.jn > 1) join(s.jn, s.j0, s.j1, s.st, single, sg);
        if (single) continue;
        s = step(sg, true, single);
        if (tid == 0) s_last[x][1] = arrive(s.cnt, s.jn);
        __syncthreads();
        if (s_last[x][1]) join(s.jn, s.j0, s.j1, s.st, true, sg);
    }
}

// the code rows of the cache: {128 bytes, 32 rows, d/128 halves of a row, pages}
static tq_status f8_page_map(CUtensorMap* m, const void* cache, int d, int64_t pages) {
    char why[200] = "";
    auto enc = tensor_map_encoder(why, sizeof why);
    if (!enc) return driver_failure("%s", why);
    const tq_status bs = bind_device_context();
    if (bs != TQ_OK) return bs;
    const cuuint64_t dims[4] = {128, 32, (cuuint64_t)(d / 128), (cuuint64_t)pages};
    const cuuint64_t strides[3] = {(cuuint64_t)d, 128, (cuuint64_t)f8_page_bytes(d)};
    const cuuint32_t box[4] = {128, 32, (cuuint32_t)(d / 128), 1}, estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(cache), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return driver_failure("cuTensorMapEncodeTiled failed (CUresult %d) for %lld pages at %p", (int)r,
                              (long long)pages, cache);
    return TQ_OK;
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
    const int grid = C::CTAS * std::min(sms, kF8MaxSms);
    CUtensorMap pages;
    st = f8_page_map(&pages, a.cache, D, a.num_blocks * a.heads);
    if (st != TQ_OK) return st;
    // launched programmatically: the launch overlaps the previous kernel's end,
    // and the kernel waits for it before its first read
    return cuda_status(launch_pdl(true, f8_decode_kernel<D, NT, PREC>, dim3(grid), dim3(kF8Threads), C::total, s, a, pages));
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
    a.gcnt = c->gcnt;
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
    // fp32 in or out: query and weights in two fp16 parts.  Up to 8 heads a unit that
    // costs nothing (8 x 20480 tokens: 63 us, 64 without); with 16, 74 us for 63 at d =
    // 128 and 96 for 62 at d = 256 (16 x 8192), so 16-bit calls do without.
    const bool prec = q_dtype == TQ_DTYPE_F32 || out_dtype == TQ_DTYPE_F32;
    cudaStream_t s = (cudaStream_t)stream;
    return d == 128 ? dispatch_f8_decode<128>(a, c->geom.nt, prec, s) : dispatch_f8_decode<256>(a, c->geom.nt, prec, s);
}
