// Prompt attention: packed query rows over packed keys and values, causal
// against the end of each sequence's keys, grouped heads.
//
//   s_ij = <q_i, k_j>;  m_i = max_j s_ij;  p_ij = 2^(c (s_ij - m_i)), c = scale log2(e)
//   out_i = sum_j p_ij v_j / sum_j p_ij;   lse_i = scale m_i + ln sum_j p_ij
//
// Bound by the tensor cores (2 d multiply-adds per query head, row and visible
// key).  A work item is 128-row query tiles of one sequence and KV head; a tile's
// rows are the G query heads of floor(128 / G) tokens, so a group shares every key
// tile and short prompts still fill the rows.  d = 128: two tiles of queries; d =
// 256: one (its output alone fills half of tensor memory); 128 keys at a time.
// (64 keys were slower at d = 256: an MMA of 64 columns takes as long as one of
// 128.)  Either way a block has two score buffers of one step each, and the tensor
// cores work on one step's products while the softmax of the other runs:
//   step i uses score buffer i & 1; d = 128: key tile i / 2 of query tile i & 1,
//   d = 256: key tile i.
//   MMA order: ... P V of step i, scores of step i + 2, P V of step i + 1, ...
// The scores of step i + 2 overwrite the probabilities of step i in place.
//
// Softmax: thread = row; its scores come from tensor memory into registers, the
// probabilities (rounded to the inputs' 16-bit type, the row sum is of the
// unrounded ones) go back as the A operand of P V.  The reference m moves only
// when it falls 2^8 behind, so that the output in tensor memory is rescaled
// rarely, and it moves a tile late: a tile's exponentials do not wait for its
// maximum, unless that lies so far ahead that they might overflow (2^14 for fp16
// probabilities, 2^20 for bf16), when they are done again.  That is exact, the
// final quotient does not depend on m.  The argument is one fma, c s - (c m), with
// c m rounded once per reference; where c m is so large that its rounding would
// count (2^12, no trained model's scores), m is subtracted from the scores first.
//
// One block per SM takes items until none is left (the first by its index, the
// next from a counter), longest first, so that the copies and score products of
// the next item run beside the output of the last.  With few items and many keys
// an item covers a part of the keys only (`parts` of them); its unnormalised
// output goes to the workspace and prompt_join_kernel adds the parts up.
//
// Measured (32/8 heads, causal, bf16; 2 d multiply-adds per visible pair): 1 x 8192,
// d = 128: 366 us, 1502 TFLOP/s (cuBLAS: 1931 in a burst); 1 x 16384: 1602; 1 x 8192,
// 32/4 heads, d = 256: 1555 to 1600; 16 prompts of up to 2048, d = 128: 218 us, 998 (an
// item of 1, 2, 4, 8, 16 key tiles takes 6.2, 8.4, 12.4, 19.2, 32.0 us: 1.6 a tile, and
// 4.6 or more beside them; masked halves of tiles do not count); 96 rows after 16384
// keys, d = 256: 48 us, 1070.
//
// Warps: 0-3 (and 4-7 at d = 128) softmax and output of query tile 0 (1), then
// one for the copies (TMA), two that issue MMAs and an idle one that completes
// the warpgroup of the register split.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "tq_device.cuh"

namespace tq {

struct PromptArgs {
    const void* v;
    int64_t v_stride;
    void* out;
    float* lse;
    const int32_t *cu_q, *cu_k;
    uint32_t *err, *next;    // next: the item counter and the count of blocks that are through
    float* part;             // parts > 1: [parts][n_q * q_heads][d] sums
    float2* meta;            //            [parts][n_q * q_heads] {m, l}
    int parts;
    int batch, n_q, n_k;
    int q_heads, heads, group, tile_tok;  // tile_tok: tokens per 128-row tile
    float scale, scale_log2;
    int causal;
};

template <int D_, bool BF16_>
struct PromptCfg {
    static constexpr int D = D_;
    static constexpr bool BF16 = BF16_;
    static constexpr int NQ = D == 128 ? 2 : 1;  // query tiles per block
    static constexpr int BN = 128;               // keys per tile
    static constexpr int EN = D / 128;           // ring entries per key or value tile
    static constexpr int CH = D / 64;            // 64-element chunks (128-byte swizzled rows)
    // bytes of a query tile and of a ring entry: 128 keys x 128 elements, or the
    // values of 128 / EN keys
    static constexpr int QB = 128 * D * 2, KB = 128 * 128 * 2, VN = BN / EN;
    static constexpr int STAGES = 5;
    // how far (log2) a score may lie above the reference before a tile is done again:
    // the probabilities' range, with room for the sums
    static constexpr float AHEAD_LOG2 = BF16 ? 20.f : 14.f;
    // from here on (log2) the rounding of c m would count: half a unit is 2^-13 here,
    // against 2^-9 and 2^-12 of a probability's
    static constexpr float FAR_LOG2 = 4096.f;
    // order of the tiles in the ring: AHEAD key tiles, then value tile 0, key tile AHEAD, value tile 1, ...
    static constexpr int AHEAD = NQ == 2 ? 1 : 2;
    static __host__ __device__ constexpr int key_pos(int j) { return j < AHEAD ? j : 2 * j - AHEAD + 1; }
    static __host__ __device__ constexpr int value_pos(int j, int n) {
        const int pos = 2 * j + AHEAD, keys_out = n - AHEAD;  // value tiles from keys_out on have no key tile between them
        return j <= keys_out ? pos : n + j;
    }
    static constexpr int SOFT = 128 * NQ;        // softmax threads
    static constexpr int THREADS = SOFT + 128;
    // tensor memory: scores (probabilities in place), then outputs
    static constexpr int COL_S = 0, COL_O = 2 * BN;
    static constexpr int off_ring = NQ * QB;
    static constexpr int off_bar = off_ring + STAGES * KB;
    static constexpr int BAR = 256;
    static constexpr int total = off_bar + BAR + 1024;  // + alignment to 1024
    static_assert(COL_O + NQ * D <= 512, "tensor memory");
    static_assert(total <= 232448, "shared memory");
};

// kind::f16 instruction descriptor: fp32 accumulators, A K-major, B K-major
// (bmn = 0) or MN-major (1), M = 128
__host__ __device__ constexpr uint32_t prompt_idesc(bool bf16, int n, int bmn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((uint32_t)bmn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// 128-byte-swizzled shared-memory operand: 8-row groups 1024 bytes apart; lbo:
// step between 64-element column blocks of an MN-major operand
__device__ __forceinline__ uint64_t prompt_desc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void prompt_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void prompt_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ float prompt_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr int kPromptParts = 16;  // key parts at most (a lane each in the join)

__device__ __forceinline__ float prompt_max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t prompt_pack(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <bool BF16>
__device__ __forceinline__ float2 prompt_values(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// pairs of fp32 (one instruction for two lanes' worth of work)
__device__ __forceinline__ uint64_t prompt_pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void prompt_unpair(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t prompt_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t prompt_add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// a wait that a stuck barrier ends once for the whole role: later waits of the
// thread are skipped and the block runs to its end
__device__ __forceinline__ void prompt_wait(uint32_t bar, uint32_t parity, bool& dead, uint32_t* err) {
    if (!dead) dead = !mbar_wait(bar, parity, err);
}

// A work item: rows [q0 + t0, ...) of a sequence, a range of its keys.
struct PromptWork {
    int ok;
    int q0, lq, k0, lk;  // first row and length of the sequence's queries and keys
    int t0;              // first token of query tile 0
    int row, part;       // KV head, part of the keys
    int j0, n[2];        // first key tile; key tiles of each query tile from there on
    int seen;            // keys that every row of the item sees; value tiles that reach behind
                         // them are checked
    __device__ __forceinline__ int tiles() const { return max(n[0], n[1]); }
    template <int BN>
    __device__ __forceinline__ bool checked(int j) const {
        return (j0 + j + 1) * BN > seen;
    }
};

// keys that token t of the sequence sees
__device__ __forceinline__ int prompt_limit(const PromptArgs& a, const PromptWork& w, int t) {
    return a.causal ? max(0, min(w.lk, t + 1 + w.lk - w.lq)) : w.lk;
}

// Item `item` (query tiles from the last on: with causal rows those have the
// most keys; KV heads and key parts of a tile side by side), run by one warp.
// `total`: the query tiles of all sequences, counted by the first call (-1).
template <class C>
__device__ __forceinline__ PromptWork prompt_find(const PromptArgs& a, int64_t item, int lane, int& total) {
    const int per = C::NQ * a.tile_tok, sub = a.heads * a.parts;
    PromptWork w;
    w.ok = 0;
    w.q0 = w.lq = w.k0 = w.lk = w.t0 = w.row = w.part = w.j0 = w.n[0] = w.n[1] = w.seen = 0;
    int have = -1, q0 = 0, q1 = 0, k0 = 0, k1 = 0;  // (up to 32 sequences are read once)
    for (int pass = total < 0 ? 0 : 1; pass < 2; ++pass) {
        int seen = 0;
        const int64_t want = (int64_t)total - 1 - item / sub;
        if (pass == 1 && want < 0) break;
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            const int b = b0 + lane;
            if (have != b0) q0 = q1 = k0 = k1 = 0;
            if (have != b0 && b < a.batch) {
                q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
                k0 = __ldg(a.cu_k + b), k1 = __ldg(a.cu_k + b + 1);
                if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_k) {
                    if (pass == 0) set_error(a.err, TQ_DEVERR_CHUNK);
                    q0 = min(max(q0, 0), a.n_q), q1 = min(max(q1, q0), a.n_q);
                    k0 = min(max(k0, 0), a.n_k), k1 = min(max(k1, k0), a.n_k);
                }
            }
            have = b0;
            const int n = (q1 - q0 + per - 1) / per;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            if (pass == 1) {
                const bool here = want >= seen + incl - n && want < seen + incl;
                const uint32_t m = __ballot_sync(0xffffffffu, here);
                if (m) {
                    const int src = __ffs(m) - 1;
                    w.ok = 1;
                    w.q0 = __shfl_sync(0xffffffffu, q0, src);
                    w.lq = __shfl_sync(0xffffffffu, q1, src) - w.q0;
                    w.k0 = __shfl_sync(0xffffffffu, k0, src);
                    w.lk = __shfl_sync(0xffffffffu, k1, src) - w.k0;
                    w.t0 = (int)(want - __shfl_sync(0xffffffffu, seen + incl - n, src)) * per;
                    break;
                }
            }
            seen += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (pass == 0) total = seen;
    }
    if (w.ok) {
        w.seen = prompt_limit(a, w, w.t0);
        const int x = (int)(item % sub);
        w.row = x / a.parts;
        w.part = x - w.row * a.parts;
        int all[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            // key tiles that the query tile's last token sees
            const int first = w.t0 + t * a.tile_tok, last = min(first + a.tile_tok, w.lq) - 1;
            all[t] = t < C::NQ && first < w.lq ? (prompt_limit(a, w, last) + C::BN - 1) / C::BN : 0;
        }
        const int most = max(all[0], all[1]);
        w.j0 = (int)((int64_t)most * w.part / a.parts);
        const int j1 = (int)((int64_t)most * (w.part + 1) / a.parts);
#pragma unroll
        for (int t = 0; t < 2; ++t) w.n[t] = max(0, min(j1, all[t]) - w.j0);
    }
    return w;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ CUtensorMap mq,
              const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    constexpr int D = C::D, NQ = C::NQ, BN = C::BN, CH = C::CH, S = C::STAGES;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::off_bar);
    const uint32_t full = smem_u32(bars), empty = full + 8 * S, qfull = empty + 8 * S, qfree = qfull + 8,
                   sfull = qfree + 8, pready = sfull + 16, pvdone = pready + 16, turn = pvdone + 16, wfull = turn + 16,
                   wfree = wfull + 16;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 2 * S + 14);
    static_assert((2 * S + 14) * 8 + 4 <= C::BAR, "barriers");
    __shared__ PromptWork s_w[2];
    __shared__ int s_bad[4];  // [it & 3] = it + 1: item it has values that are not finite in its checked rows
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int W0 = C::SOFT / 32;  // first of the other four warps: copies, MMA
    uint32_t* err = a.err;

    if (tid < 4) s_bad[tid] = 0;
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, NQ);
        }
        mbar_init(qfull, 1);
        mbar_init(qfree, NQ);
        for (int t = 0; t < 2; ++t) {
            mbar_init(sfull + 8 * t, 1);
            mbar_init(pready + 8 * t, 4);
            mbar_init(pvdone + 8 * t, 1);
            mbar_init(turn + 8 * t, 1);
            mbar_init(wfull + 8 * t, 1);
            mbar_init(wfree + 8 * t, 2 + W0);  // the issuing threads and the softmax warps
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // launched programmatically: what is above overlaps the previous kernel's end (not
    // the allocation, which could take tensor memory that kernel still asks for)
    pdl_wait();
    if (warp == 0) tmem_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    bool dead = false;
    // Every role walks the same items; what it counts over them (ring positions,
    // uses of a score buffer) gives the parities of its waits.
    int ring = 0, use0 = 0, use1 = 0;
    auto advance = [&](const PromptWork& w) {
        ring += 2 * C::EN * w.tiles();
        use0 += NQ == 2 ? w.n[0] : (w.tiles() + 1) / 2;
        use1 += NQ == 2 ? w.n[1] : w.tiles() / 2;
    };
    // item number `it` of this block
    auto fetch = [&](int it, PromptWork& w) {
        prompt_wait(wfull + 8 * (it & 1), (it >> 1) & 1, dead, err);
        w = s_w[it & 1];
        if (dead) w.ok = 0;
    };

    if (warp >= W0) {
        if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(56));
        if (warp == W0) {
            // ---------------------------------------------------- copies
            int total = -1, loads = 0, q_loads = 0;
            int64_t item = blockIdx.x;
            for (int it = 0;; ++it) {
                const PromptWork w = prompt_find<C>(a, item, lane, total);
                if (it >= 2) prompt_wait(wfree + 8 * (it & 1), ((it >> 1) - 1) & 1, dead, err);
                __syncwarp();
                if (lane == 0) {
                    s_w[it & 1] = w;
                    mbar_arrive(wfull + 8 * (it & 1));
                }
                if (!w.ok) break;
                const int n = w.tiles();
                if (lane == 0 && n > 0 && !dead) {
                    if (q_loads > 0) prompt_wait(qfree, (q_loads - 1) & 1, dead, err);
                    if (!dead) {
                        ++q_loads;
                        // the tokens of both tiles that exist (rows of others come along and are not used)
                        const int tiles = NQ == 2 && w.n[1] > 0 ? 2 : 1;
                        mbar_expect_tx(qfull, (uint32_t)(tiles * CH * a.tile_tok * a.group * 128));
                        for (int t = 0; t < tiles; ++t)
                            for (int c = 0; c < CH; ++c)
                                tma_4d(smem_u32(smem) + t * C::QB + c * (128 * 128), &mq, 64 * c, 0, w.row,
                                       w.q0 + w.t0 + t * a.tile_tok, qfull);
                    }
                    // a key tile goes in by halves of the elements, a value tile by
                    // halves of the keys (at d = 128 either in one piece)
                    auto load = [&](bool key, int j) {
                        for (int h = 0; h < C::EN; ++h) {
                            const int s = loads % S;
                            if (loads >= S) prompt_wait(empty + 8 * s, ((loads / S) - 1) & 1, dead, err);
                            if (dead) return;
                            const uint32_t dst = smem_u32(smem) + C::off_ring + s * C::KB;
                            const int k0 = w.k0 + (w.j0 + j) * BN;
                            mbar_expect_tx(full + 8 * s, C::KB);
                            if (key)
                                for (int c = 0; c < 2; ++c)
                                    tma_3d(dst + c * (BN * 128), &mk, 64 * (2 * h + c), w.row, k0, full + 8 * s);
                            else
                                for (int c = 0; c < CH; ++c)
                                    tma_3d(dst + c * (C::VN * 128), &mv, 64 * c, w.row, k0 + h * C::VN, full + 8 * s);
                            ++loads;
                        }
                    };
                    for (int j = 0; j < C::AHEAD && j < n; ++j) load(true, j);
                    for (int j = 0; j < n; ++j) {
                        load(false, j);
                        if (j + C::AHEAD < n) load(true, j + C::AHEAD);
                    }
                }
                __syncwarp();
                // the next item: asked for when this one's copies are under way (not
                // before: who is through first shall have the longest that is left)
                uint32_t next = 0;
                if (lane == 0) next = atomicAdd(a.next, 1u);
                dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
                item = (int64_t)gridDim.x + __shfl_sync(0xffffffffu, next, 0);
            }
            if (lane == 0) {
                // copies still in flight land before the block exits
                if (dead) {
                    bool d2 = false;
                    for (int i = max(0, loads - S); i < loads; ++i) prompt_wait(full + 8 * (i % S), (i / S) & 1, d2, err);
                    d2 = false;
                    if (q_loads > 0) prompt_wait(qfull, (q_loads - 1) & 1, d2, err);
                }
                // the last block leaves the counters ready for the next call
                if (atomicAdd(a.next + 1, 1u) == gridDim.x - 1) a.next[0] = a.next[1] = 0;
            }
        } else if (warp <= W0 + 2) {
            // -------------------------------------------------------- MMA
            // Two issuing threads, so that the waits of one are hidden behind the
            // products of the other (a wait and the first MMA after it cost about
            // 165 cycles, and the tensor cores queue only two or three MMAs of 64).
            // d = 128: one per query tile; they take turns, so that one tile's
            // products run beside the other's softmax.  d = 256: one for the
            // scores, one for the value products.
            if (lane == 0) {
                constexpr uint32_t id_s = prompt_idesc(C::BF16, BN, 0), id_o = prompt_idesc(C::BF16, D, 1);
                const int me = warp - (W0 + 1);
                const uint64_t q_desc = prompt_desc(smem_u32(smem), 16);
                const uint64_t k_desc = prompt_desc(smem_u32(smem) + C::off_ring, 16);
                const uint64_t v_desc = prompt_desc(smem_u32(smem) + C::off_ring, C::VN * 128);
                auto take = [&](int pos, int h) {  // entry h of the tile at `pos` of the item's ring order
                    const int r = ring + C::EN * pos + h;
                    prompt_wait(full + 8 * (r % S), (r / S) & 1, dead, err);
                    return r % S;
                };
                // element half h of a key tile.  `early` runs before the last three
                // MMAs: what it lets another thread issue lines up behind them
                auto scores = [&](int buf, int t, int s, int h, auto early) {
                    const uint64_t qd = q_desc + (uint64_t)((t * C::QB + h * 2 * (128 * 128)) >> 4);
                    const uint64_t kd = k_desc + (uint64_t)(s * (C::KB >> 4));
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (k == 8 - 3) early();
                        prompt_mma_ss(tmem + C::COL_S + buf * BN,
                                      qd + (uint64_t)(((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                                      kd + (uint64_t)(((k >> 2) * (BN * 128) + (k & 3) * 32) >> 4), id_s, h > 0 || k > 0);
                    }
                    if (h == C::EN - 1) tc_commit(sfull + 8 * buf);
                };
                // key half h of a value tile (at d = 256)
                auto values = [&](int buf, int t, int s, int h, bool first) {
                    const uint64_t vd = v_desc + (uint64_t)(s * (C::KB >> 4));
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < C::VN / 16; ++k)
                        prompt_mma_ts(tmem + C::COL_O + t * D, tmem + C::COL_S + buf * BN + 8 * (h * (C::VN / 16) + k),
                                      vd + (uint64_t)((k * 2048) >> 4), id_o, !(first && h == 0 && k == 0));
                    if (h == C::EN - 1) tc_commit(pvdone + 8 * buf);
                };
                int q_uses = 0, turns = 0;
                PromptWork w;
                for (int it = 0;; ++it) {
                    fetch(it, w);
                    mbar_arrive(wfree + 8 * (it & 1));
                    if (!w.ok) break;
                    const int n = w.tiles();
                    if (n == 0) continue;
                    auto value_tile = [&](int j, int h) { return take(C::value_pos(j, n), h); };
                    if constexpr (NQ == 2) {
                        // both threads see every ring position and release every stage
                        const int mine = me == 0 ? w.n[0] : w.n[1], use = me == 0 ? use0 : use1;
                        const bool both = w.n[0] > 0 && w.n[1] > 0;
                        auto begin = [&]() {
                            if (!both) return;
                            if (me == 1 || turns > 0) prompt_wait(turn + 8 * me, (turns - (me == 0)) & 1, dead, err);
                            ++turns;
                        };
                        auto pass = [&]() {
                            if (both) mbar_arrive(turn + 8 * (1 - me));
                        };
                        prompt_wait(qfull, q_uses & 1, dead, err);
                        int ks = take(C::key_pos(0), 0);
                        begin();
                        if (mine > 0) scores(me, me, ks, 0, pass);
                        else pass();
                        tc_commit(empty + 8 * ks);
                        if (mine <= 1) tc_commit(qfree);
                        for (int j = 0; j < n; ++j) {
                            const int vs = value_tile(j, 0);
                            if (j + 1 < n) ks = take(C::key_pos(j + 1), 0);
                            begin();
                            if (j < mine) prompt_wait(pready + 8 * me, (use + j) & 1, dead, err);
                            if (j < mine) values(me, me, vs, 0, j == 0);
                            // (these scores overwrite the probabilities, whose products this
                            // thread issued before: MMAs of a thread run in order)
                            if (j + 1 < mine) scores(me, me, ks, 0, pass);
                            else pass();
                            tc_commit(empty + 8 * vs);
                            if (j + 1 < n) tc_commit(empty + 8 * ks);
                            if (j + 2 == mine) tc_commit(qfree);  // the tile's last scores are issued
                        }
                    } else if (me == 0) {
                        // A thread that comes to a ring position has seen what orders the
                        // stage's earlier phases before it: here the value products of the
                        // buffer's last use, below the probabilities of the tile.
                        prompt_wait(qfull, q_uses & 1, dead, err);
                        for (int j = 0; j < n; ++j) {
                            // the buffer's probabilities are used up
                            const int use = (j & 1 ? use1 : use0) + (j >> 1);
                            if (use > 0) prompt_wait(pvdone + 8 * (j & 1), (use - 1) & 1, dead, err);
                            for (int h = 0; h < C::EN; ++h) {
                                const int ks = take(C::key_pos(j), h);
                                scores(j & 1, 0, ks, h, [] {});
                                tc_commit(empty + 8 * ks);
                            }
                        }
                        tc_commit(qfree);
                    } else {
                        for (int j = 0; j < n; ++j) {
                            const int use = (j & 1 ? use1 : use0) + (j >> 1);
                            prompt_wait(pready + 8 * (j & 1), use & 1, dead, err);
                            for (int h = 0; h < C::EN; ++h) {
                                const int vs = value_tile(j, h);
                                values(j & 1, 0, vs, h, j == 0);
                                tc_commit(empty + 8 * vs);
                            }
                        }
                    }
                    ++q_uses;
                    advance(w);
                }
            }
        }
    } else {
        // ------------------------------------------------ softmax, output
        if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(224));
        const int t = NQ == 2 ? warp >> 2 : 0;
        const int rt = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int tt = rt / a.group, head = rt - tt * a.group;
        const uint32_t so = tmem + lanes + C::COL_O + t * D;
        const float c = a.scale_log2;
        PromptWork w;
        for (int it = 0;; ++it) {
            fetch(it, w);
            __syncwarp();
            if (lane == 0) mbar_arrive(wfree + 8 * (it & 1));
            if (!w.ok) break;
            const int nt = t == 0 ? w.n[0] : w.n[1], first = w.t0 + t * a.tile_tok, tok = first + tt;
            const bool live = rt < a.tile_tok * a.group && tok < w.lq;
            const int lim = live ? prompt_limit(a, w, tok) : 0;
            // key tiles that every row of the tile sees whole
            const int whole = prompt_limit(a, w, min(first, w.lq)) / BN;
            const int64_t row = (int64_t)(w.q0 + tok) * a.q_heads + w.row * a.group + head;
            // A probability of zero does not keep a value out of a product: 0 * inf
            // and 0 * NaN are NaN.  In a value tile with rows that some query row does
            // not see, the rows behind the sequence's last key (a neighbour's) become
            // zero, and so do values that are not finite in rows that only some query
            // rows see; the output adds those to the rows that see them.  Done before
            // the tile's probabilities are signalled, by the query tile's four warps.
            // (At d = 128 both query tiles do it; what one has zeroed the other finds
            // zero, and the flag set before.)
            auto check = [&](int j) {
                const uint32_t em = C::BF16 ? 0x7F807F80u : 0x7C007C00u, e1 = C::BF16 ? 0x00800080u : 0x04000400u;
                if (NQ == 1 && j > 0) {
                    // (orders the ring's earlier phases before the wait below)
                    const int pb = (j - 1) & 1;
                    prompt_wait(pvdone + 8 * pb, ((pb ? use1 : use0) + ((j - 1) >> 1)) & 1, dead, err);
                }
                bool wrote = false;
#pragma unroll 1
                for (int h = 0; h < C::EN; ++h) {
                    const int r = ring + C::EN * C::value_pos(j, w.tiles()) + h, key0 = (w.j0 + j) * BN + h * C::VN;
                    // A wait on `full` tells this load from the stage's last one only when
                    // that one is known to be there.  The tile before this one, or the last
                    // item's, says so; at d = 128 a query tile without keys in the last item
                    // has waited for nothing in it.  What made the stage free for this load
                    // does: both issuing threads had taken the load before.
                    if (NQ == 2 && j == 0 && r >= S) prompt_wait(empty + 8 * (r % S), (r / S - 1) & 1, dead, err);
                    prompt_wait(full + 8 * (r % S), (r / S) & 1, dead, err);
                    uint8_t* v = smem + C::off_ring + (r % S) * C::KB;
                    // rows [r0, r1) to check, [r1, VN) to zero, in CH columns of 128
                    // bytes; 8 lanes a row, 16 rows at a time
                    const int r1 = max(0, min(C::VN, w.lk - key0)), r0 = min(r1, max(0, w.seen - key0));
                    auto at = [&](int c, int rr) { return reinterpret_cast<uint4*>(v + (c * C::VN + rr) * 128 + (rt & 7) * 16); };
                    auto inf = [&](uint32_t y) { return (y & em) + e1; };  // bits 15, 31: not finite
                    uint32_t any = 0;
#pragma unroll 1
                    for (int rr = r0 + (rt >> 3); rr < r1; rr += 64) {
                        uint4 x[4][2];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                x[u][c] = rr + 16 * u < r1 ? *at(c, rr + 16 * u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
#pragma unroll
                            for (int c = 0; c < 2; ++c) any |= inf(x[u][c].x) | inf(x[u][c].y) | inf(x[u][c].z) | inf(x[u][c].w);
                        if constexpr (CH > 2) {
#pragma unroll
                            for (int u = 0; u < 4; ++u)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    x[u][c] = rr + 16 * u < r1 ? *at(c + 2, rr + 16 * u) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                            for (int u = 0; u < 4; ++u)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    any |= inf(x[u][c].x) | inf(x[u][c].y) | inf(x[u][c].z) | inf(x[u][c].w);
                        }
                    }
                    if (any & 0x80008000u) {
                        s_bad[it & 3] = it + 1;
                        __threadfence_block();
                        wrote = true;
#pragma unroll 1
                        for (int c = 0; c < CH; ++c)
#pragma unroll 1
                            for (int rr = r0 + (rt >> 3); rr < r1; rr += 16) {
                                auto fix = [&](uint32_t y) {
                                    const uint32_t f = inf(y);
                                    return y & ~((f & 0x8000u ? 0xFFFFu : 0u) | (f & 0x80000000u ? 0xFFFF0000u : 0u));
                                };
                                const uint4 x = *at(c, rr);
                                *at(c, rr) = make_uint4(fix(x.x), fix(x.y), fix(x.z), fix(x.w));
                            }
                    }
                    if (r1 < C::VN) {
                        wrote = true;
#pragma unroll 1
                        for (int c = 0; c < CH; ++c)
#pragma unroll 1
                            for (int rr = r1 + (rt >> 3); rr < C::VN; rr += 16) *at(c, rr) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                // (the other query tile's warps may have written what this one reads)
                __threadfence_block();
                if (wrote || s_bad[it & 3] == it + 1) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            };
            auto rescale = [&](int j, float f) {  // the output's sums, before tile j's
                if (j == 0) return;
                if constexpr (NQ == 1) {
                    // the products of the tile before, of the other buffer
                    const int pb = (j - 1) & 1;
                    prompt_wait(pvdone + 8 * pb, ((pb ? use1 : use0) + ((j - 1) >> 1)) & 1, dead, err);
                    tc_fence_after();
                }
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    tmem_ld32(so + i, o);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st32(so + i, o);
                }
            };
            float m = -INFINITY, l = 0.f, mx = -INFINITY;
            bool far = false;  // a row of the warp has a reference beyond FAR_LOG2
            int j = 0;
            for (; j < nt; ++j) {
                const int buf = NQ == 2 ? t : j & 1, use = (buf ? use1 : use0) + (NQ == 2 ? j : j >> 1);
                const uint32_t ss = tmem + lanes + C::COL_S + buf * BN;
                // (while the scores are under way; at d = 256 the wait for the values
                // needs the scores before it)
                if (NQ == 2 && w.checked<BN>(j)) check(j);
                prompt_wait(sfull + 8 * buf, use & 1, dead, err);
                tc_fence_after();
                uint32_t s[BN / 32][32];
#pragma unroll
                for (int i = 0; i < BN / 32; ++i) tmem_ld32(ss + 32 * i, s[i]);
                tc_wait_ld();
                if (w.j0 + j >= whole) {
                    const int cut = lim - (w.j0 + j) * BN;
#pragma unroll
                    for (int i = 0; i < BN / 32; ++i)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * i + k >= cut) s[i][k] = 0xFF800000u;
                }
                float xa = -INFINITY, xb = -INFINITY;  // maximum of the tile
                auto chunk_max = [&](int i) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        xa = prompt_max3(xa, __uint_as_float(s[i][k]), __uint_as_float(s[i][k + 1]));
                        xb = prompt_max3(xb, __uint_as_float(s[i][k + 2]), __uint_as_float(s[i][k + 3]));
                    }
                };
                // a tile row that no token of the sequence has (its queries are a neighbour's, or
                // what shared memory held) has no say in what its warp does
                auto row_max = [&]() { return live ? prompt_max3(mx, xa, xb) : -INFINITY; };
                if (j == 0) {
#pragma unroll
                    for (int i = 0; i < BN / 32; ++i) chunk_max(i);
                    mx = row_max();
                }
                float lj = 0.f;
                bool again = false;
                do {
                    // the first time's rescaled output and probabilities are there before the
                    // output is read once more
                    if (again) tc_wait_st();
                    // mx: the maximum up to the last tile (the first time), or up to this one
                    const bool move = (mx - m) * c > 8.f;  // also from -inf to the first score
                    if (__any_sync(0xffffffffu, move)) {
                        const float f = !move ? 1.f : m == -INFINITY ? 0.f : prompt_exp2((m - mx) * c);
                        if (move) m = mx;
                        l *= f;
                        rescale(j, f);
                        far = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m) * c > C::FAR_LOG2);
                        if (far) break;
                    }
                    const float mc = m == -INFINITY ? 0.f : m * c;
                    const uint64_t c2 = prompt_pair(c, c), mc2 = prompt_pair(-mc, -mc);
                    uint64_t la = 0, lb = 0;  // sums of even and odd pairs
                    // groups of four scores in three stages (argument; exponential;
                    // sum, rounding, maximum), a group apart, so that the
                    // exponentials, 4 cycles each, have the rest in their shadow
                    uint64_t arg[2][2];
                    float x[2][4];
                    uint32_t p[16];
#pragma unroll
                    for (int g = 0; g < BN / 4 + 2; ++g) {
                        if (g < BN / 4) {
                            const uint32_t* v = &s[g >> 3][4 * (g & 7)];
                            arg[g & 1][0] = prompt_fma2(prompt_pair(__uint_as_float(v[0]), __uint_as_float(v[1])), c2, mc2);
                            arg[g & 1][1] = prompt_fma2(prompt_pair(__uint_as_float(v[2]), __uint_as_float(v[3])), c2, mc2);
                        }
                        if (g >= 1 && g <= BN / 4) {
                            float* y = x[(g - 1) & 1];
                            prompt_unpair(arg[(g - 1) & 1][0], y[0], y[1]);
                            prompt_unpair(arg[(g - 1) & 1][1], y[2], y[3]);
#pragma unroll
                            for (int u = 0; u < 4; ++u) y[u] = prompt_exp2(y[u]);
                        }
                        if (g >= 2) {
                            const int h = g - 2;
                            const float* y = x[h & 1];
                            const uint32_t* v = &s[h >> 3][4 * (h & 7)];
                            la = prompt_add2(la, prompt_pair(y[0], y[1]));
                            lb = prompt_add2(lb, prompt_pair(y[2], y[3]));
                            p[2 * (h & 7)] = prompt_pack<C::BF16>(y[0], y[1]);
                            p[2 * (h & 7) + 1] = prompt_pack<C::BF16>(y[2], y[3]);
                            xa = prompt_max3(xa, __uint_as_float(v[0]), __uint_as_float(v[1]));
                            xb = prompt_max3(xb, __uint_as_float(v[2]), __uint_as_float(v[3]));
                            if ((h & 7) == 7) tmem_st16(ss + 16 * (h >> 3), p);
                        }
                    }
                    float x0, x1;
                    prompt_unpair(prompt_add2(la, lb), x0, x1);
                    lj = x0 + x1;
                    if (again) break;
                    mx = row_max();
                    again = __any_sync(0xffffffffu, (mx - m) * c > C::AHEAD_LOG2);
                } while (again);
                if (far) {
                    // the loop below takes over; it reads the scores once more
                    if (again) {
#pragma unroll
                        for (int i = 0; i < BN / 32; ++i) tmem_st32(ss + 32 * i, s[i]);
                    }
                    tc_wait_st();
                    break;
                }
                l += lj;
                if (NQ == 1 && w.checked<BN>(j)) check(j);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready + 8 * buf);
            }
            // Scores this large: the reference is subtracted before they are scaled.  From the
            // tile on in which the first such reference was taken, without the head start on
            // the maximum and without haste: two passes over the scores in tensor memory.
#pragma unroll 1
            for (; j < nt; ++j) {
                const int buf = NQ == 2 ? t : j & 1, use = (buf ? use1 : use0) + (NQ == 2 ? j : j >> 1);
                const uint32_t ss = tmem + lanes + C::COL_S + buf * BN;
                prompt_wait(sfull + 8 * buf, use & 1, dead, err);
                tc_fence_after();
                if (w.checked<BN>(j)) check(j);
                const int cut = live ? lim - (w.j0 + j) * BN : 0;
                uint32_t y[32], p[16];
#pragma unroll 1
                for (int i = 0; i < BN; i += 32) {
                    tmem_ld32(ss + i, y);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (i + k < cut) mx = fmaxf(mx, __uint_as_float(y[k]));
                }
                const bool move = (mx - m) * c > 8.f;
                if (__any_sync(0xffffffffu, move)) {
                    const float f = !move ? 1.f : m == -INFINITY ? 0.f : prompt_exp2((m - mx) * c);
                    if (move) m = mx;
                    l *= f;
                    rescale(j, f);
                }
                const float by = m == -INFINITY ? 0.f : m;
                float lj = 0.f;
#pragma unroll 1
                for (int i = 0; i < BN; i += 32) {
                    tmem_ld32(ss + i, y);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float e0 = i + k < cut ? prompt_exp2((__uint_as_float(y[k]) - by) * c) : 0.f;
                        const float e1 = i + k + 1 < cut ? prompt_exp2((__uint_as_float(y[k + 1]) - by) * c) : 0.f;
                        lj += e0 + e1;
                        p[k / 2] = prompt_pack<C::BF16>(e0, e1);
                    }
                    tmem_st16(ss + i / 2, p);
                }
                l += lj;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready + 8 * buf);
            }
            if (nt > 0) {
                const int buf = NQ == 2 ? t : (nt - 1) & 1, use = (buf ? use1 : use0) + (NQ == 2 ? nt - 1 : (nt - 1) >> 1);
                prompt_wait(pvdone + 8 * buf, use & 1, dead, err);
                tc_fence_after();
            }
            if (nt > 0 && s_bad[it & 3] == it + 1) {
                // the values that were left out of the products, to the rows that see
                // them (into the sums in tensor memory; rare, so it may take its time)
                const int last = min(lim, (w.j0 + nt) * BN);
#pragma unroll 1
                for (int i = 0; i < D; i += 16) {
                    uint32_t o[16];
                    tmem_ld16(so + i, o);
                    tc_wait_ld();
#pragma unroll 1
                    for (int key = max(w.seen, w.j0 * BN); key < last; ++key) {
                        const uint32_t* v = reinterpret_cast<const uint32_t*>(
                            static_cast<const uint16_t*>(a.v) + (int64_t)(w.k0 + key) * a.v_stride + w.row * D + i);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 x = prompt_values<C::BF16>(__ldg(v + k));
                            if (!isfinite(x.x)) o[2 * k] = __float_as_uint(__uint_as_float(o[2 * k]) + x.x);
                            if (!isfinite(x.y)) o[2 * k + 1] = __float_as_uint(__uint_as_float(o[2 * k + 1]) + x.y);
                        }
                    }
                    __syncwarp();
                    tmem_st16(so + i, o);
                }
                tc_wait_st();
            }
            // 4 x 4 transposition over a quad of lanes: swap pieces with lane ^ 1, then with
            // lane ^ 2; lane u of a quad ends up with 16-byte piece u of the quad's four rows
            const int u = lane & 3;
            auto quad = [&](uint32_t (&p)[4][4]) {
#pragma unroll
                for (int b = 1; b < 4; b <<= 1)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (!(q & b))
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const uint32_t send = u & b ? p[q][x] : p[q | b][x];
                                const uint32_t got = __shfl_xor_sync(0xffffffffu, send, b);
                                if (u & b) p[q][x] = got;
                                else p[q | b][x] = got;
                            }
            };
            // four lanes write 64 bytes of one row side by side (a lane alone would touch
            // 32 lines with every store)
            int64_t rows[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) rows[r] = __shfl_sync(0xffffffffu, live ? row : -1, (lane & ~3) + r);
            if (a.parts > 1) {
                const int64_t part = (int64_t)w.part * a.n_q * a.q_heads;
                if (nt > 0) {
#pragma unroll 1
                    for (int i = 0; i < D; i += 16) {
                        uint32_t o[16];
                        tmem_ld16(so + i, o);
                        tc_wait_ld();
                        uint32_t p[4][4];
#pragma unroll
                        for (int k = 0; k < 16; ++k) p[k >> 2][k & 3] = o[k];
                        quad(p);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (rows[r] >= 0)
                                *reinterpret_cast<uint4*>(a.part + (part + rows[r]) * D + i + 4 * u) =
                                    make_uint4(p[r][0], p[r][1], p[r][2], p[r][3]);
                    }
                }
                if (live) a.meta[part + row] = make_float2(m, l);
            } else {
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    if (nt > 0) {
                        tmem_ld32(so + i, o);
                        tc_wait_ld();
                    }
                    uint32_t p[4][4];  // [piece][word]
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        p[k >> 2][k & 3] = l == 0.f ? 0u
                                                    : prompt_pack<C::BF16>(__uint_as_float(o[2 * k]) * inv,
                                                                           __uint_as_float(o[2 * k + 1]) * inv);
                    quad(p);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (rows[r] >= 0)
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + rows[r] * D + i + 8 * u) =
                                make_uint4(p[r][0], p[r][1], p[r][2], p[r][3]);
                }
                if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
            }
            // (the next item's first value products wait for its probabilities,
            // which this warp signals after these reads of the output)
            advance(w);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// Add the parts of every row up, one warp per row and head; a part without a key of
// the row has l = 0 and no sums.  Eight parts' loads are under way at a time.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ PromptArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t rows = (int64_t)a.n_q * a.q_heads, row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_wait();
    if (row >= rows) return;
    // rows no sequence names are left as they were
    const int tok = (int)(row / a.q_heads);
    bool mine = false;
    for (int b = lane; b < a.batch; b += 32) mine |= __ldg(a.cu_q + b) <= tok && tok < __ldg(a.cu_q + b + 1);
    // lane z: part z
    const float2 ml = lane < a.parts ? __ldcg(a.meta + lane * rows + row) : make_float2(-INFINITY, 0.f);
    if (!__any_sync(0xffffffffu, mine)) return;
    const float M = warp_max(ml.x);
    const float f = ml.y == 0.f ? 0.f : M == -INFINITY ? 1.f : prompt_exp2((ml.x - M) * a.scale_log2);
    const float l = warp_sum(ml.y == 0.f ? 0.f : ml.y * f);
    const uint32_t there = __ballot_sync(0xffffffffu, ml.y != 0.f);
    float o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    for (int z0 = 0; z0 < a.parts; z0 += 8) {
        float4 x[8][D / 128];
#pragma unroll
        for (int z = 0; z < 8; ++z)
#pragma unroll
            for (int i = 0; i < D / 128; ++i)
                if (there >> (z0 + z) & 1)
                    x[z][i] = __ldcg(reinterpret_cast<const float4*>(a.part + ((z0 + z) * rows + row) * D) + lane + 32 * i);
#pragma unroll
        for (int z = 0; z < 8; ++z) {
            const float fz = __shfl_sync(0xffffffffu, f, z0 + z);
            if (there >> (z0 + z) & 1)
#pragma unroll
                for (int i = 0; i < D / 128; ++i) {
                    o[4 * i] = fmaf(x[z][i].x, fz, o[4 * i]), o[4 * i + 1] = fmaf(x[z][i].y, fz, o[4 * i + 1]);
                    o[4 * i + 2] = fmaf(x[z][i].z, fz, o[4 * i + 2]), o[4 * i + 3] = fmaf(x[z][i].w, fz, o[4 * i + 3]);
                }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < D / 128; ++i)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + 128 * i + 4 * lane) =
            make_uint2(prompt_pack<BF16>(o[4 * i] * inv, o[4 * i + 1] * inv),
                       prompt_pack<BF16>(o[4 * i + 2] * inv, o[4 * i + 3] * inv));
    if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : M * a.scale + logf(l);
}

// Parts of the keys: as many as shorten the longest run of a block, the join
// (about 5 us) counted in (96 rows after 16384 keys, 24 items: 271 us in one part, 48
// in six; 8192 rows are not cut).  The lengths are on the device; what the host knows is
// the row counts.
template <class C>
int prompt_parts(const PromptArgs& a, int64_t items, int sms, int64_t part_rows) {
    const double keys = (double)a.n_k - (a.causal ? 0.5 * std::min(a.n_q, a.n_k) : 0.0);
    const double tiles = keys / a.batch / C::BN, tile_us = 1.7;
    int best = 1;
    double best_us = 0;
    for (int z = 1; z <= kPromptParts; ++z) {
        if (z > 1 && ((int64_t)z * a.n_q * a.q_heads > part_rows || tiles < 2 * z)) break;
        const double waves = (double)((items * z + sms - 1) / sms);
        const double us = waves * (tiles / z * tile_us + 2.0) + (z > 1 ? 5.0 + 0.3 * z : 0.0);
        if (z == 1 || us < 0.95 * best_us) best = z, best_us = us;
    }
    return best;
}

template <class C>
tq_status launch_prompt(PromptArgs a, int64_t part_rows, const CUtensorMap& mq, const CUtensorMap& mk,
                        const CUtensorMap& mv, cudaStream_t s) {
    int sms = 0;
    tq_status st = device_sms(&sms);
    if (st == TQ_OK) st = ensure_dynamic_smem((const void*)prompt_kernel<C>, C::total, "prompt_kernel");
    if (st != TQ_OK) return st;
    // at most this many items: the last tile of every sequence may be short of rows
    const int per = C::NQ * a.tile_tok;
    const int64_t items = ((int64_t)a.n_q + (int64_t)a.batch * (per - 1)) / per * a.heads;
    a.parts = prompt_parts<C>(a, items, sms, part_rows);
    const int grid = (int)std::min<int64_t>(items * a.parts, sms);
    st = cuda_status(launch_pdl(true, prompt_kernel<C>, dim3(grid), dim3(C::THREADS), C::total, s, a, mq, mk, mv));
    if (st == TQ_OK && a.parts > 1)
        st = cuda_status(launch_pdl(true, prompt_join_kernel<C::D, C::BF16>, dim3((unsigned)(((int64_t)a.n_q * a.q_heads + 7) / 8)), dim3(256), 0, s, a));
    return st;
}

tq_status launch_prompt_128(const PromptArgs& a, int64_t part_rows, const CUtensorMap& mq, const CUtensorMap& mk,
                            const CUtensorMap& mv, bool bf16, cudaStream_t s);
tq_status launch_prompt_256(const PromptArgs& a, int64_t part_rows, const CUtensorMap& mq, const CUtensorMap& mk,
                            const CUtensorMap& mv, bool bf16, cudaStream_t s);

}  // namespace tq
