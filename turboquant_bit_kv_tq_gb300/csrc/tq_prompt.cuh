// Prompt attention: packed query rows over packed keys and values, causal
// against the end of each sequence's keys, grouped heads.
//
//   s_ij = <q_i, k_j>;  m_i = max_j s_ij;  p_ij = 2^(c (s_ij - m_i)), c = scale log2(e)
//   out_i = sum_j p_ij v_j / sum_j p_ij;   lse_i = scale m_i + ln sum_j p_ij
//
// Bound by the tensor cores (4 d multiply-adds per query head, row and visible
// key, times 2 flops).  A block takes 128-row query tiles of one sequence and KV
// head; a tile's rows are the G query heads of floor(128 / G) tokens, so a group
// shares every key tile and short prompts still fill the rows.  d = 128: two
// tiles of queries, 128 keys at a time; d = 256: one tile, 64 keys at a time
// (its output alone fills half of tensor memory).  Either way a block has two
// score buffers of one step each, and the tensor cores work on one step's
// products while the softmax of the other runs:
//   step i uses score buffer i & 1; d = 128: key tile i / 2 of query tile i & 1,
//   d = 256: key tile i.
//   MMA order: ... P V of step i, scores of step i + 2, P V of step i + 1, ...
// The scores of step i + 2 overwrite the probabilities of step i in place.
//
// Softmax: thread = row; its scores come from tensor memory into registers, the
// probabilities (rounded to the inputs' 16-bit type, the row sum is of the
// unrounded ones) go back as the A operand of P V, in two halves of the keys so
// that the products of the first run beside the exponentials of the second.  The reference m moves only
// when it falls 2^8 behind, so that the output in tensor memory is rescaled
// rarely; that is exact, the final quotient does not depend on m.
//
// Warps: 0-3 (and 4-7 at d = 128) softmax and output of query tile 0 (1), then
// one for the copies (TMA), two that issue MMAs and an idle one that completes
// the warpgroup of the register split.
#pragma once

#include <cuda.h>

#include "tq_device.cuh"

namespace tq {

struct PromptArgs {
    const void* q;
    int64_t q_stride;
    void* out;
    float* lse;
    const int32_t *cu_q, *cu_k;
    uint32_t* err;
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
    static constexpr int BN = D == 128 ? 128 : 64;
    static constexpr int CH = D / 64;            // 64-element chunks (128-byte swizzled rows)
    static constexpr int QB = 128 * D * 2, KB = BN * D * 2;  // bytes of a query / key tile
    // d = 256: the query tile goes to tensor memory (the score products' shared-memory
    // traffic, 6 KB per MMA of 32 cycles with both operands there, would bound them)
    static constexpr bool QT = D == 256;
    static constexpr int STAGES = QT ? 7 : 5;
    // ring order: AHEAD key tiles, then value tile 0, key tile AHEAD, value tile 1, ...
    static constexpr int AHEAD = NQ == 2 ? 1 : 2;
    static __host__ __device__ constexpr int key_pos(int j) { return j < AHEAD ? j : 2 * j - AHEAD + 1; }
    static __host__ __device__ constexpr int value_pos(int j, int n) {
        const int pos = 2 * j + AHEAD, keys_out = n - AHEAD;  // value tiles from keys_out on have no key tile between them
        return j <= keys_out ? pos : n + j;
    }
    static constexpr int SOFT = 128 * NQ;        // softmax threads
    static constexpr int THREADS = SOFT + 128;
    // tensor memory: scores (probabilities in place), then outputs
    static constexpr int COL_S = 0, COL_O = 2 * BN, COL_Q = COL_O + NQ * D;
    static constexpr int off_ring = QT ? 0 : NQ * QB;
    static constexpr int off_bar = off_ring + STAGES * KB;
    static constexpr int total = off_bar + 256 + 1024;  // + alignment to 1024
    static_assert(COL_Q + (QT ? D / 2 : 0) <= 512, "tensor memory");
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

// What a block works on: rows [q0 + t0, ...) of a sequence, its keys.
struct PromptWork {
    int ok;
    int q0, lq, k0, lk;  // first row and length of the sequence's queries and keys
    int t0;              // first token of query tile 0
    int n[2];            // key tiles of each query tile
    int row;             // KV head
};

// keys that token t of the sequence sees
__device__ __forceinline__ int prompt_limit(const PromptArgs& a, const PromptWork& w, int t) {
    return a.causal ? max(0, min(w.lk, t + 1 + w.lk - w.lq)) : w.lk;
}

// Work item `item` of the sequences' query tiles (the last first: with causal
// rows those have the most keys), run by one warp.
template <class C>
__device__ __forceinline__ PromptWork prompt_find(const PromptArgs& a, int item, int lane) {
    const int per = C::NQ * a.tile_tok;
    PromptWork w;
    w.ok = 0;
    int total = 0;
    // total first, then the item counted from the end
    for (int pass = 0; pass < 2; ++pass) {
        int seen = 0;
        const int want = total - 1 - item;
        if (pass == 1 && want < 0) break;
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            const int b = b0 + lane;
            int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
            if (b < a.batch) {
                q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
                k0 = __ldg(a.cu_k + b), k1 = __ldg(a.cu_k + b + 1);
                if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_k) {
                    if (pass == 0) set_error(a.err, TQ_DEVERR_CHUNK);
                    q0 = min(max(q0, 0), a.n_q), q1 = min(max(q1, q0), a.n_q);
                    k0 = min(max(k0, 0), a.n_k), k1 = min(max(k1, k0), a.n_k);
                }
            }
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
                    w.t0 = (want - __shfl_sync(0xffffffffu, seen + incl - n, src)) * per;
                    return w;
                }
            }
            seen += __shfl_sync(0xffffffffu, incl, 31);
        }
        total = seen;
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
    const uint32_t full = smem_u32(bars), empty = full + 8 * S, qfull = empty + 8 * S, sfull = qfull + 8,
                   pready = sfull + 16, pvdone = pready + 32, vclean = pvdone + 16, turn = vclean + 8;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 2 * S + 12);
    __shared__ PromptWork s_w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int W0 = C::SOFT / 32;  // first of the other four warps: copies, MMA
    uint32_t* err = a.err;

    if (warp == W0) {
        PromptWork w = prompt_find<C>(a, blockIdx.x / a.heads, lane);
        if (w.ok) {
            w.row = blockIdx.x % a.heads;
            for (int t = 0; t < 2; ++t) {
                // keys that the tile's last token sees
                const int first = w.t0 + t * a.tile_tok, last = min(first + a.tile_tok, w.lq) - 1;
                w.n[t] = t < NQ && first < w.lq ? (prompt_limit(a, w, last) + BN - 1) / BN : 0;
            }
        }
        if (lane == 0) {
            s_w = w;
            for (int s = 0; s < S; ++s) {
                mbar_init(full + 8 * s, 1);
                mbar_init(empty + 8 * s, NQ);
            }
            mbar_init(qfull, C::QT ? 4 : 1);
            for (int t = 0; t < 2; ++t) {
                mbar_init(sfull + 8 * t, 1);
                mbar_init(pready + 16 * t, 4);  // the first and the second half of the keys
                mbar_init(pready + 16 * t + 8, 4);
                mbar_init(pvdone + 8 * t, 1);
                mbar_init(turn + 8 * t, 1);
            }
            mbar_init(vclean, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    if (warp == 0) tmem_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const PromptWork w = s_w;
    const int n0 = w.ok ? w.n[0] : 0, n1 = w.ok && NQ == 2 ? w.n[1] : 0, n = max(n0, n1);
    bool dead = false;

    if (warp >= W0) {
        if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(72));
        if (warp == W0) {
            // ---------------------------------------------------- copies
            if (lane == 0 && n > 0) {
                // the tokens of both tiles that exist (rows of others come along and are not used)
                if constexpr (!C::QT) {
                    const int tiles = NQ == 2 && n1 > 0 ? 2 : 1;
                    mbar_expect_tx(qfull, (uint32_t)(tiles * CH * a.tile_tok * a.group * 128));
                    for (int t = 0; t < tiles; ++t)
                        for (int c = 0; c < CH; ++c)
                            tma_4d(smem_u32(smem) + t * C::QB + c * (128 * 128), &mq, 64 * c, 0, w.row,
                                   w.q0 + w.t0 + t * a.tile_tok, qfull);
                }
                int r = 0;
                auto load = [&](const CUtensorMap* m, int j) {
                    const int s = r % S;
                    if (r >= S) prompt_wait(empty + 8 * s, ((r / S) - 1) & 1, dead, err);
                    if (!dead) {
                        mbar_expect_tx(full + 8 * s, C::KB);
                        for (int c = 0; c < CH; ++c)
                            tma_3d(smem_u32(smem) + C::off_ring + s * C::KB + c * (BN * 128), m, 64 * c, w.row,
                                   w.k0 + j * BN, full + 8 * s);
                        ++r;
                    }
                };
                for (int j = 0; j < C::AHEAD && j < n; ++j) load(&mk, j);
                for (int j = 0; j < n; ++j) {
                    load(&mv, j);
                    if (j + C::AHEAD < n) load(&mk, j + C::AHEAD);
                }
                // copies still in flight land before the block exits
                if (dead) {
                    bool d2 = false;
                    for (int i = max(0, r - S); i < r; ++i) prompt_wait(full + 8 * (i % S), (i / S) & 1, d2, err);
                    d2 = false;
                    if (!C::QT) prompt_wait(qfull, 0, d2, err);
                }
            }
            // zero the value rows behind the sequence's last key: 0 * NaN or inf
            // of a neighbour's row would be NaN.  The last value tile was the
            // last copy, the 2 n-th of the ring.
            __syncwarp();
            dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
            if (n > 0 && w.lk % BN != 0 && w.lk / BN == n - 1) {
                const int s = (2 * n - 1) % S;
                prompt_wait(full + 8 * s, ((2 * n - 1) / S) & 1, dead, err);
                uint8_t* v = smem + C::off_ring + s * C::KB;
                for (int i = lane; i < CH * BN * 8; i += 32)
                    if ((i >> 3) % BN >= w.lk % BN) *reinterpret_cast<uint4*>(v + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(vclean);
            }
        } else if (warp <= W0 + 2) {
            // -------------------------------------------------------- MMA
            // Two issuing threads, so that the waits of one are hidden behind the
            // products of the other (a wait and the first MMA after it cost about
            // 165 cycles, and the tensor cores queue only two or three MMAs of 64).
            // d = 128: one per query tile; they take turns, so that one tile's
            // products run beside the other's softmax.  d = 256: one for the
            // scores, one for the value products.
            if (lane == 0 && n > 0) {
                constexpr uint32_t id_s = prompt_idesc(C::BF16, BN, 0), id_o = prompt_idesc(C::BF16, D, 1);
                const int me = warp - (W0 + 1);
                const uint64_t q_desc = prompt_desc(smem_u32(smem), 16);
                const uint64_t k_desc = prompt_desc(smem_u32(smem) + C::off_ring, 16);
                const uint64_t v_desc = prompt_desc(smem_u32(smem) + C::off_ring, BN * 128);
                auto take = [&](int r) {  // ring position r
                    prompt_wait(full + 8 * (r % S), (r / S) & 1, dead, err);
                    return r % S;
                };
                auto scores = [&](int buf, int t, int s) {
                    const uint64_t qd = q_desc + (uint64_t)(t * (C::QB >> 4));
                    const uint64_t kd = k_desc + (uint64_t)(s * (C::KB >> 4));
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                    {
                        const uint64_t b = kd + (uint64_t)(((k >> 2) * (BN * 128) + (k & 3) * 32) >> 4);
                        if constexpr (C::QT)
                            prompt_mma_ts(tmem + C::COL_S + buf * BN, tmem + C::COL_Q + 8 * k, b, id_s, k > 0);
                        else
                            prompt_mma_ss(tmem + C::COL_S + buf * BN,
                                          qd + (uint64_t)(((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4), b, id_s, k > 0);
                    }
                    tc_commit(sfull + 8 * buf);
                };
                auto values = [&](int buf, int t, int s, bool first, uint32_t parity) {
                    const uint64_t vd = v_desc + (uint64_t)(s * (C::KB >> 4));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (NQ == 1) prompt_wait(pready + 16 * buf + 8 * h, parity, dead, err);
                        tc_fence_after();
#pragma unroll
                        for (int k = h * BN / 32; k < (h + 1) * BN / 32; ++k)
                            prompt_mma_ts(tmem + C::COL_O + t * D, tmem + C::COL_S + buf * BN + 8 * k,
                                          vd + (uint64_t)((k * 2048) >> 4), id_o, !(first && k == 0));
                    }
                    tc_commit(pvdone + 8 * buf);
                };
                const bool ragged = w.lk % BN != 0;
                auto value_tile = [&](int r, int j) {
                    const int s = take(r);
                    if (ragged && j == w.lk / BN) prompt_wait(vclean, 0, dead, err);
                    return s;
                };
                if constexpr (NQ == 2) {
                    // both threads see every ring position and release every stage
                    const int mine = me == 0 ? n0 : n1;
                    const bool both = n0 > 0 && n1 > 0;
                    int turns = 0;
                    auto begin = [&]() {
                        if (both && (me == 1 || turns > 0)) prompt_wait(turn + 8 * me, (turns - (me == 0)) & 1, dead, err);
                        ++turns;
                    };
                    auto pass = [&]() {
                        if (both) mbar_arrive(turn + 8 * (1 - me));
                    };
                    prompt_wait(qfull, 0, dead, err);
                    int ks = take(C::key_pos(0));
                    begin();
                    if (mine > 0) scores(me, me, ks);
                    pass();
                    tc_commit(empty + 8 * ks);
                    for (int j = 0; j < n; ++j) {
                        const int vs = value_tile(C::value_pos(j, n), j);
                        if (j + 1 < n) ks = take(C::key_pos(j + 1));
                        if (j < mine) prompt_wait(pready + 16 * me + 8, j & 1, dead, err);
                        begin();
                        if (j < mine) values(me, me, vs, j == 0, j & 1);
                        // (these scores overwrite the probabilities, whose products this
                        // thread issued before: MMAs of a thread run in order)
                        if (j + 1 < mine) scores(me, me, ks);
                        pass();
                        tc_commit(empty + 8 * vs);
                        if (j + 1 < n) tc_commit(empty + 8 * ks);
                    }
                } else if (me == 0) {
                    // A thread that comes to a ring position has seen what orders the
                    // stage's earlier phases before it: here the value products of tile
                    // j - 2, below the probabilities of tile j.
                    prompt_wait(qfull, 0, dead, err);
                    for (int j = 0; j < n; ++j) {
                        // the buffer's probabilities are used up
                        if (j >= 2) prompt_wait(pvdone + 8 * (j & 1), ((j >> 1) - 1) & 1, dead, err);
                        const int ks = take(C::key_pos(j));
                        scores(j & 1, 0, ks);
                        tc_commit(empty + 8 * ks);
                    }
                } else {
                    for (int j = 0; j < n; ++j) {
                        prompt_wait(pready + 16 * (j & 1), (j >> 1) & 1, dead, err);
                        const int vs = value_tile(C::value_pos(j, n), j);
                        values(j & 1, 0, vs, j == 0, (j >> 1) & 1);
                        tc_commit(empty + 8 * vs);
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------ softmax, output
        if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(216));
        const int t = NQ == 2 ? warp >> 2 : 0;
        const int rt = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int nt = t == 0 ? n0 : n1;
        const int tok = w.t0 + t * a.tile_tok + rt / a.group, head = rt % a.group;
        const bool live = w.ok && rt < a.tile_tok * a.group && tok < w.lq;
        const int lim = live ? prompt_limit(a, w, tok) : 0;
        // key tiles that every row of the tile sees whole
        const int whole = w.ok ? prompt_limit(a, w, min(w.t0 + t * a.tile_tok, w.lq)) / BN : 0;
        const uint32_t so = tmem + lanes + C::COL_O + t * D;
        const float c = a.scale_log2;
        if constexpr (C::QT) {
            if (n > 0) {
                const uint4* q = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(a.q) + (live ? (int64_t)(w.q0 + tok) * a.q_stride + (int64_t)(w.row * a.group + head) * D : 0));
#pragma unroll 1
                for (int i = 0; i < D / 64; ++i) {
                    uint32_t x[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 v = live ? __ldg(q + 8 * i + k) : make_uint4(0u, 0u, 0u, 0u);
                        x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
                    }
                    tmem_st32(tmem + lanes + C::COL_Q + 32 * i, x);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(qfull);
            }
        }
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < nt; ++j) {
            const int buf = NQ == 2 ? t : j & 1;
            const uint32_t ss = tmem + lanes + C::COL_S + buf * BN;
            prompt_wait(sfull + 8 * buf, (NQ == 2 ? j : j >> 1) & 1, dead, err);
            tc_fence_after();
            uint32_t s[BN / 32][32];
#pragma unroll
            for (int i = 0; i < BN / 32; ++i) tmem_ld32(ss + 32 * i, s[i]);
            tc_wait_ld();
            if (j >= whole) {
                const int cut = lim - j * BN;
#pragma unroll
                for (int i = 0; i < BN / 32; ++i)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (32 * i + k >= cut) s[i][k] = 0xFF800000u;
            }
            float mx = -INFINITY, mx2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < BN / 32; ++i)
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    mx = fmaxf(mx, fmaxf(__uint_as_float(s[i][k]), __uint_as_float(s[i][k + 1])));
                    mx2 = fmaxf(mx2, fmaxf(__uint_as_float(s[i][k + 2]), __uint_as_float(s[i][k + 3])));
                }
            mx = fmaxf(mx, mx2);
            const bool move = (mx - m) * c > 8.f;  // also from -inf to the first score
            if (__any_sync(0xffffffffu, move)) {
                const float f = !move ? 1.f : m == -INFINITY ? 0.f : prompt_exp2((m - mx) * c);
                if (move) m = mx;
                l *= f;
                if (j > 0) {
                    if constexpr (NQ == 1) {
                        prompt_wait(pvdone + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, dead, err);
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
                }
            }
            const float mc = m == -INFINITY ? 0.f : m * c;
            const uint64_t c2 = prompt_pair(c, c), mc2 = prompt_pair(-mc, -mc);
            uint64_t la = 0, lb = 0;  // sums of even and odd pairs
#pragma unroll
            for (int i = 0; i < BN / 32; ++i) {
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    float x[4];
                    prompt_unpair(prompt_fma2(prompt_pair(__uint_as_float(s[i][k]), __uint_as_float(s[i][k + 1])), c2, mc2),
                                  x[0], x[1]);
                    prompt_unpair(prompt_fma2(prompt_pair(__uint_as_float(s[i][k + 2]), __uint_as_float(s[i][k + 3])), c2, mc2),
                                  x[2], x[3]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[u] = prompt_exp2(x[u]);
                    la = prompt_add2(la, prompt_pair(x[0], x[1]));
                    lb = prompt_add2(lb, prompt_pair(x[2], x[3]));
                    p[k / 2] = prompt_pack<C::BF16>(x[0], x[1]);
                    p[k / 2 + 1] = prompt_pack<C::BF16>(x[2], x[3]);
                }
                tmem_st16(ss + 16 * i, p);
                if (i == BN / 64 - 1 || i == BN / 32 - 1) {
                    // half of the keys: their value products may start
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pready + 16 * buf + (i == BN / 32 - 1 ? 8 : 0));
                }
            }
            {
                float x0, x1;
                prompt_unpair(prompt_add2(la, lb), x0, x1);
                l += x0 + x1;
            }
        }
        if (nt > 0) {
            if constexpr (NQ == 2) prompt_wait(pvdone + 8 * t, (nt - 1) & 1, dead, err);
            else prompt_wait(pvdone + 8 * ((nt - 1) & 1), ((nt - 1) >> 1) & 1, dead, err);
            tc_fence_after();
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t row = (int64_t)(w.q0 + tok) * a.q_heads + w.row * a.group + head;
        uint16_t* out = static_cast<uint16_t*>(a.out) + row * D;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            if (nt > 0) {
                tmem_ld32(so + i, o);
                tc_wait_ld();
            }
            if (live) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t p[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        p[u] = l == 0.f ? 0u
                                        : prompt_pack<C::BF16>(__uint_as_float(o[k + 2 * u]) * inv,
                                                               __uint_as_float(o[k + 2 * u + 1]) * inv);
                    *reinterpret_cast<uint4*>(out + i + k) = make_uint4(p[0], p[1], p[2], p[3]);
                }
            }
        }
        if (live && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <class C>
tq_status launch_prompt(const PromptArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                        cudaStream_t s) {
    const tq_status st = ensure_dynamic_smem((const void*)prompt_kernel<C>, C::total, "prompt_kernel");
    if (st != TQ_OK) return st;
    // every sequence's last block may be short of rows; blocks without work return at once
    const int64_t items = (int64_t)a.n_q / (C::NQ * a.tile_tok) + a.batch;
    if (items * a.heads > 0x7FFFFFFF) return TQ_ERR_INVALID_ARG;
    prompt_kernel<C><<<(unsigned)(items * a.heads), C::THREADS, C::total, s>>>(a, mq, mk, mv);
    return cuda_status(cudaGetLastError());
}

tq_status launch_prompt_128(const PromptArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                            bool bf16, cudaStream_t s);
tq_status launch_prompt_256(const PromptArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                            bool bf16, cudaStream_t s);

}  // namespace tq
