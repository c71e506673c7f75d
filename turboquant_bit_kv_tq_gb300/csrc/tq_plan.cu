// The plan of a step: block-table entries, slots, positions and row starts of a
// batch's new tokens.
//
// Every block sums up all requests (8 KB of lengths for 1024 of them, from L2) and keeps
// the sums in shared memory; then a thread takes a token, finds its request by
// bisection and writes the token's entries.  The token in the first row of a block
// writes the block's entry of the table: each new block has exactly one.  Bound by
// latency: lengths, sums, bisection, block id, one dependent step after the other.

#include <algorithm>
#include <new>

#include "tq_device.cuh"

struct tq_plan {
    tq_plan_config cfg;
    uint32_t *err, *cnt;
};

namespace tq {

struct PlanArgs {
    const int32_t *lens, *fresh, *free, *next;
    int32_t* table;
    int64_t* slots;
    int32_t *pos, *rows, *seq_lens, *cu_q, *cu_k, *next_out;
    uint32_t *err, *cnt;
    int batch, columns, n_free, n_tokens;
    bool in_place;  // an output is an input's memory
};

constexpr int kPlanThreads = 256, kPlanWarps = kPlanThreads / 32, kPlanMaxBatch = 8192, kPlanTokens = 256;

// what a block keeps beside its sums
struct PlanShared {
    int64_t scan[kPlanWarps][3];
    bool last;
};
// The launch limit without an opt-in is 48 KB of both together
constexpr int kPlanOptIn = 47 * 1024;
static_assert(sizeof(PlanShared) <= 1024 - 64, "shared memory beside the sums");

// inclusive sums over the block's threads of N values; tot: those of all
template <int N>
__device__ __forceinline__ void plan_scan(int64_t (&x)[N], int64_t (&tot)[N], int64_t (*s)[3]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t up = __shfl_up_sync(0xffffffffu, x[k], o);
            if (lane >= o) x[k] += up;
        }
    __syncthreads();
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < N; ++k) s[warp][k] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int64_t before = 0;
        tot[k] = 0;
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            const int64_t v = s[w][k];
            if (w < warp) before += v;
            tot[k] += v;
        }
        x[k] += before;
    }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int32_t sm[];
    // per request: first row, stored tokens, tokens served, its blocks' place in the list
    int32_t *s_cu = sm, *s_len = s_cu + a.batch + 1, *s_served = s_len + a.batch, *s_off = s_served + a.batch;
    int32_t* s_row = s_off + a.batch;  // first row of packed keys (all new tokens have one, served or not)
    __shared__ PlanShared sh;
    const int tid = threadIdx.x;
    const int64_t cap = (int64_t)a.columns * 16;
    pdl_wait();  // (the launch overlaps the previous kernel's end)
    int next = *a.next;  // (plain loads of what the last block may overwrite)
    uint32_t bad = 0;
    if (next < 0 || next > a.n_free) bad |= TQ_DEVERR_POOL, next = max(0, min(next, a.n_free));
    const int64_t avail = a.n_free - next;

    // a request's stored and new tokens, within their limits
    auto request = [&](int b, int64_t& len, int64_t& n) {
        len = n = 0;
        if (b >= a.batch) return;
        len = a.lens[b];
        n = a.fresh ? a.fresh[b] : 1;
        if (len < 0 || len > cap || n < 0) bad |= TQ_DEVERR_SEQLEN;
        len = max((int64_t)0, min(len, cap));
        n = max((int64_t)0, n);
    };
    // Requests in chunks of one per thread.  First as if all rows and blocks sufficed: one
    // sum of rows, blocks and keys.  If they do not, again, one after the other: a
    // request's rows depend on the rows before it, its blocks on its rows.
    int64_t rows0 = 0, blocks0 = 0, keys0 = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int64_t len, n;
        request(b, len, n);
        const int64_t served = min(n, cap - len), want = ((len + served + 15) >> 4) - ((len + 15) >> 4);
        int64_t x[3] = {n, want, len + n}, tot[3];
        plan_scan(x, tot, sh.scan);
        if (b < a.batch) {
            if (served < n) bad |= TQ_DEVERR_SEQLEN;
            s_cu[b] = (int)min((int64_t)0x7FFFFFFF, rows0 + x[0] - n);
            s_len[b] = (int)len;
            s_served[b] = (int)served;
            s_off[b] = (int)min((int64_t)0x7FFFFFFF, blocks0 + x[1] - want);
            s_row[b] = (int)min((int64_t)0x7FFFFFFF, keys0 + x[2] - len - n);
        }
        rows0 += tot[0], blocks0 += tot[1], keys0 += tot[2];
    }
    if (rows0 > a.n_tokens || blocks0 > avail) {
        rows0 = blocks0 = keys0 = 0;
        bad &= ~TQ_DEVERR_SEQLEN;  // (found again, for the rows there are)
        for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
            const int b = b0 + tid;
            int64_t len, n;
            request(b, len, n);
            int64_t x[1] = {n}, tot[1], both[2];
            plan_scan(x, tot, sh.scan);
            const int64_t first = min((int64_t)a.n_tokens, rows0 + x[0] - n);
            if (rows0 + x[0] > a.n_tokens) bad |= TQ_DEVERR_CHUNK;
            rows0 += tot[0];
            n = min(n, a.n_tokens - first);
            if (n > cap - len) bad |= TQ_DEVERR_SEQLEN;
            int64_t served = min(n, cap - len);
            const int64_t have = (len + 15) >> 4;
            const int64_t want = ((len + served + 15) >> 4) - have;
            int64_t y[2] = {want, len + n};
            plan_scan(y, both, sh.scan);
            const int64_t off = blocks0 + y[0] - want;
            blocks0 += both[0];
            if (off + want > avail) {
                bad |= TQ_DEVERR_POOL;
                served = min(served, 16 * (have + max((int64_t)0, avail - off)) - len);
            }
            if (b < a.batch) {
                s_cu[b] = (int)first;
                s_len[b] = (int)len;
                s_served[b] = (int)served;
                s_off[b] = (int)min(off, (int64_t)0x7FFFFFFF);
                s_row[b] = (int)min((int64_t)0x7FFFFFFF, keys0 + y[1] - len - n);
            }
            keys0 += both[1];
        }
    }
    const int rows = (int)min(rows0, (int64_t)a.n_tokens);
    if (tid == 0) s_cu[a.batch] = rows;
    __syncthreads();

    for (int64_t t = (int64_t)blockIdx.x * kPlanThreads + tid; t < a.n_tokens; t += (int64_t)gridDim.x * kPlanThreads) {
        int64_t slot = -1;
        int pos = 0, row = -1;
        if (t < rows) {
            // the last request whose first row is not behind t
            int lo = 0, hi = a.batch;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int i = (int)t - s_cu[lo], len = s_len[lo];
            pos = (int)min((uint32_t)len + (uint32_t)i, 0x7FFFFFFFu);  // (far behind the widest row's end)
            if (i < s_served[lo]) {
                row = (int)min((uint32_t)s_row[lo] + (uint32_t)pos, 0x7FFFFFFFu);
                const int col = pos >> 4, have = (len + 15) >> 4;
                int32_t* entry = a.table + (int64_t)lo * a.columns + col;
                int id;
                if (col >= have) {
                    id = __ldg(a.free + next + s_off[lo] + (col - have));
                    if ((pos & 15) == 0) *entry = id;
                } else {
                    id = *entry;
                }
                if (id >= 0) slot = (int64_t)id * 16 + (pos & 15);
            }
        }
        a.slots[t] = slot;
        a.pos[t] = pos;
        a.rows[t] = row;
    }
    if (bad) set_error(a.err, bad);

    // lengths and list entry: by the first block, or, where they are the inputs' memory, by
    // the last to arrive, when every block has read them
    if (a.in_place && gridDim.x > 1) {
        if (tid == 0) {
            __threadfence();
            sh.last = atomicAdd(a.cnt, 1u) == gridDim.x - 1;
            if (sh.last) *a.cnt = 0;
        }
        __syncthreads();
        if (!sh.last) return;
    } else if (blockIdx.x > 0) {
        return;
    }
    for (int b = tid; b < a.batch; b += kPlanThreads) {
        a.seq_lens[b] = s_len[b] + s_served[b];
        a.cu_q[b] = s_cu[b];
        a.cu_k[b] = s_row[b];
    }
    if (tid == 0) {
        a.cu_q[a.batch] = rows;
        a.cu_k[a.batch] = (int)min((int64_t)0x7FFFFFFF, keys0);
        *a.next_out = next + (int)min(blocks0, avail);
    }
}

static bool plan_overlap(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
    return (uintptr_t)a < (uintptr_t)(b + m) && (uintptr_t)b < (uintptr_t)(a + n);
}

static tq_status plan_check(const tq_plan_config& c) {
    if (c.max_batch < 1 || c.max_blocks_per_seq < 1) return TQ_ERR_INVALID_ARG;
    if (c.max_batch > kPlanMaxBatch) return TQ_ERR_UNSUPPORTED;
    if ((double)c.max_batch * c.max_blocks_per_seq * 16 > 2147483647.0) return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_plan_sizes(const tq_plan_config* cfg, size_t* workspace_bytes) {
    if (!cfg) return TQ_ERR_INVALID_ARG;
    const tq_status st = plan_check(*cfg);
    if (st != TQ_OK) return st;
    if (workspace_bytes) *workspace_bytes = 16;
    return TQ_OK;
}

tq_status tq_plan_create(const tq_plan_config* cfg, void* workspace_dev, void* stream, tq_plan** out) {
    if (!cfg || !workspace_dev || !out) return TQ_ERR_INVALID_ARG;
    *out = nullptr;
    const tq_status st = plan_check(*cfg);
    if (st != TQ_OK) return st;
    if ((uintptr_t)workspace_dev & 15) return TQ_ERR_MISALIGNED;
    tq_plan* h = new (std::nothrow) tq_plan();
    if (!h) return TQ_ERR_INVALID_ARG;
    h->cfg = *cfg;
    h->err = static_cast<uint32_t*>(workspace_dev);
    h->cnt = h->err + 1;
    cudaStream_t s = (cudaStream_t)stream;
    tq_status cs = cuda_status(cudaMemsetAsync(workspace_dev, 0, 16, s));
    if (cs == TQ_OK) cs = cuda_status(cudaStreamSynchronize(s));
    if (cs != TQ_OK) {
        delete h;
        return cs;
    }
    *out = h;
    return TQ_OK;
}

tq_status tq_plan_destroy(tq_plan* plan) {
    delete plan;
    return TQ_OK;
}

tq_status tq_plan_step(const tq_plan* p, const int32_t* lens, const int32_t* new_lens, int batch,
                       const int32_t* free_blocks, int64_t num_free, const int32_t* next_free, int32_t* block_table,
                       int64_t num_tokens, int64_t* slot_mapping, int32_t* positions, int32_t* kv_rows,
                       int32_t* seq_lens, int32_t* cu_q, int32_t* cu_k, int32_t* next_free_out, void* stream) {
    if (!p || batch < 1 || batch > p->cfg.max_batch) return TQ_ERR_INVALID_ARG;
    if (num_tokens < 0 || num_tokens > 0x7FFFFFFF || num_free < 0 || num_free > 0x7FFFFFFF) return TQ_ERR_INVALID_ARG;
    if (!lens || !next_free || !block_table || !seq_lens || !cu_q || !cu_k || !next_free_out || (!free_blocks && num_free > 0) ||
        (num_tokens > 0 && (!slot_mapping || !positions || !kv_rows)))
        return TQ_ERR_INVALID_ARG;
    if ((((uintptr_t)lens | (uintptr_t)new_lens | (uintptr_t)free_blocks | (uintptr_t)next_free | (uintptr_t)block_table |
          (uintptr_t)positions | (uintptr_t)kv_rows | (uintptr_t)seq_lens | (uintptr_t)cu_q | (uintptr_t)cu_k |
          (uintptr_t)next_free_out) & 3) || ((uintptr_t)slot_mapping & 7))
        return TQ_ERR_MISALIGNED;
    PlanArgs a;
    a.lens = lens, a.fresh = new_lens, a.free = free_blocks, a.next = next_free;
    a.table = block_table;
    a.slots = slot_mapping;
    a.pos = positions, a.rows = kv_rows;
    a.seq_lens = seq_lens, a.cu_q = cu_q, a.cu_k = cu_k, a.next_out = next_free_out;
    a.err = p->err, a.cnt = p->cnt;
    a.batch = batch;
    a.columns = p->cfg.max_blocks_per_seq;
    a.n_free = (int)num_free;
    a.n_tokens = (int)num_tokens;
    a.in_place = plan_overlap(seq_lens, batch, lens, batch) || plan_overlap(next_free_out, 1, next_free, 1) ||
                 (new_lens && plan_overlap(seq_lens, batch, new_lens, batch)) ||
                 plan_overlap(seq_lens, batch, next_free, 1) || plan_overlap(next_free_out, 1, lens, batch);
    int sms = 0;
    tq_status st = device_sms(&sms);
    if (st != TQ_OK) return st;
    const int smem = (5 * batch + 1) * 4;
    if (smem > kPlanOptIn) {
        st = ensure_dynamic_smem((const void*)plan_kernel, (5 * kPlanMaxBatch + 1) * 4, "plan_kernel");
        if (st != TQ_OK) return st;
    }
    // (64 requests, 59000 tokens: 1024 tokens a block 4.6 us, 256 3.2 us, 128 3.4 us)
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((num_tokens + kPlanTokens - 1) / kPlanTokens, 4 * (int64_t)sms));
    return cuda_status(launch_pdl(true, plan_kernel, dim3(grid), dim3(kPlanThreads), smem, (cudaStream_t)stream, a));
}

tq_status tq_plan_get_device_error(const tq_plan* p, uint32_t* flags, void* stream) {
    if (!p || !flags) return TQ_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    uint32_t v = 0;
    tq_status st = cuda_status(cudaMemcpyAsync(&v, p->err, 4, cudaMemcpyDeviceToHost, s));
    if (st == TQ_OK) st = cuda_status(cudaMemsetAsync(p->err, 0, 4, s));
    if (st == TQ_OK) st = cuda_status(cudaStreamSynchronize(s));
    if (st == TQ_OK) *flags = v;
    return st;
}

}  // extern "C"
