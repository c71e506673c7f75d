// Prompt attention: handle, argument checks and tensor maps.

#include <algorithm>
#include <cmath>
#include <new>

#include "tq_prompt.cuh"
#include "tq_tma.h"

struct tq_prompt {
    tq_prompt_config cfg;
    uint32_t *err, *next;
    float* part;
    float2* meta;
    int64_t part_rows;
};

namespace tq {

static tq_status prompt_check(const tq_prompt_config& c) {
    if (c.head_dim != 128 && c.head_dim != 256) return TQ_ERR_UNSUPPORTED;
    if (c.dtype != TQ_DTYPE_BF16 && c.dtype != TQ_DTYPE_F16) return TQ_ERR_UNSUPPORTED;
    if (c.num_kv_heads < 1 || c.num_q_heads < c.num_kv_heads || c.num_q_heads % c.num_kv_heads) return TQ_ERR_INVALID_ARG;
    if (c.num_q_heads / c.num_kv_heads > 128) return TQ_ERR_UNSUPPORTED;
    if (c.max_batch < 1 || c.max_tokens < 1) return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

// The workspace: error word and item counters (256 bytes), then the sums and
// {m, l} of part_rows rows: what two waves of kPromptSms blocks with full items (128
// rows at d = 256, 256 at d = 128) can write, or 16 parts of the most rows if that is
// less.  A call is cut into z parts only while z times its rows fit (prompt_parts);
// items that are not full can be more than two waves of blocks.
constexpr int kPromptSms = 160;
static int64_t prompt_part_rows(const tq_prompt_config& c) {
    const int64_t all = (int64_t)kPromptParts * c.max_tokens * c.num_q_heads;
    return std::min<int64_t>(all, 2 * kPromptSms * (c.head_dim == 128 ? 256 : 128));
}
static size_t prompt_meta_off(const tq_prompt_config& c) {
    return 256 + (size_t)prompt_part_rows(c) * c.head_dim * 4;
}

// 16-bit rows [n][heads][d] `stride` elements apart as a map over (d, [group,]
// heads, n) with a box of 64 elements (one 128-byte swizzled row) x [group x] 1 x rows
static tq_status prompt_map(CUtensorMap* m, const void* base, bool bf16, int d, int group, int heads, int64_t n,
                            int64_t stride, int rows) {
    char why[200] = "";
    auto enc = tensor_map_encoder(why, sizeof why);
    if (!enc) return driver_failure("%s", why);
    const tq_status bs = bind_device_context();
    if (bs != TQ_OK) return bs;
    const bool q = group > 0;
    const int g = q ? group : 1;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)(q ? g : heads), (cuuint64_t)(q ? heads : n), (cuuint64_t)n};
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)(q ? (int64_t)g * d * 2 : stride * 2),
                                   (cuuint64_t)stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(q ? g : 1), (cuuint32_t)(q ? 1 : rows), (cuuint32_t)rows};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, q ? 4 : 3,
                           const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return driver_failure("cuTensorMapEncodeTiled failed (CUresult %d) for %lld rows at %p, stride %lld", (int)r,
                              (long long)n, base, (long long)stride);
    return TQ_OK;
}

}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_prompt_sizes(const tq_prompt_config* cfg, size_t* workspace_bytes) {
    if (!cfg) return TQ_ERR_INVALID_ARG;
    const tq_status st = prompt_check(*cfg);
    if (st == TQ_OK && workspace_bytes) *workspace_bytes = prompt_meta_off(*cfg) + (size_t)prompt_part_rows(*cfg) * 8;
    return st;
}

tq_status tq_prompt_create(const tq_prompt_config* cfg, void* workspace_dev, void* stream, tq_prompt** out) {
    if (!cfg || !workspace_dev || !out) return TQ_ERR_INVALID_ARG;
    *out = nullptr;
    const tq_status st = prompt_check(*cfg);
    if (st != TQ_OK) return st;
    if ((uintptr_t)workspace_dev & 15) return TQ_ERR_MISALIGNED;
    tq_prompt* h = new (std::nothrow) tq_prompt();
    if (!h) return TQ_ERR_INVALID_ARG;
    h->cfg = *cfg;
    uint8_t* ws = static_cast<uint8_t*>(workspace_dev);
    h->err = reinterpret_cast<uint32_t*>(ws);
    h->next = h->err + 2;
    h->part = reinterpret_cast<float*>(ws + 256);
    h->meta = reinterpret_cast<float2*>(ws + prompt_meta_off(*cfg));
    h->part_rows = prompt_part_rows(*cfg);
    cudaStream_t s = (cudaStream_t)stream;
    tq_status cs = cuda_status(cudaMemsetAsync(workspace_dev, 0, 256, s));
    if (cs == TQ_OK) cs = cuda_status(cudaStreamSynchronize(s));
    if (cs != TQ_OK) {
        delete h;
        return cs;
    }
    *out = h;
    return TQ_OK;
}

tq_status tq_prompt_destroy(tq_prompt* p) {
    delete p;
    return TQ_OK;
}

tq_status tq_prompt_attention(const tq_prompt* p, const void* q, const void* k, const void* v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k,
                              int batch, int n_q, int n_k, float scale, int causal, void* out, float* lse,
                              void* stream) {
    if (!p || n_q < 0 || n_k < 0) return TQ_ERR_INVALID_ARG;
    const tq_prompt_config& c = p->cfg;
    if (batch < 1 || batch > c.max_batch || n_q > c.max_tokens) return TQ_ERR_INVALID_ARG;
    if (n_q == 0) return TQ_OK;
    if (!q || !cu_q || !cu_k || !out || (n_k > 0 && (!k || !v))) return TQ_ERR_INVALID_ARG;
    const int d = c.head_dim;
    if (q_stride < (int64_t)c.num_q_heads * d || (n_k > 0 && (k_stride < (int64_t)c.num_kv_heads * d ||
                                                              v_stride < (int64_t)c.num_kv_heads * d)))
        return TQ_ERR_INVALID_ARG;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)(q_stride * 2)) & 15) return TQ_ERR_MISALIGNED;
    if (n_k > 0 && (((uintptr_t)k | (uintptr_t)v | (uintptr_t)(k_stride * 2) | (uintptr_t)(v_stride * 2)) & 15))
        return TQ_ERR_MISALIGNED;
    if (n_k == 0) {  // no key anywhere: nothing of these is read
        k = v = q;
        k_stride = v_stride = q_stride;
    }
    PromptArgs a;
    a.v = v;
    a.v_stride = v_stride;
    a.out = out;
    a.lse = lse;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.err = p->err;
    a.next = p->next;
    a.part = p->part;
    a.meta = p->meta;
    a.parts = 1;
    a.batch = batch;
    a.n_q = n_q;
    a.n_k = n_k;
    a.q_heads = c.num_q_heads;
    a.heads = c.num_kv_heads;
    a.group = c.num_q_heads / c.num_kv_heads;
    a.tile_tok = 128 / a.group;
    a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d);
    a.scale_log2 = a.scale * 1.4426950408889634f;
    a.causal = causal != 0;
    const bool bf16 = c.dtype == TQ_DTYPE_BF16;
    CUtensorMap mq, mk, mv;
    tq_status st = prompt_map(&mq, q, bf16, d, a.group, a.heads, n_q, q_stride, a.tile_tok);
    if (st == TQ_OK) st = prompt_map(&mk, k, bf16, d, 0, a.heads, n_k > 0 ? n_k : n_q, k_stride, 128);
    if (st == TQ_OK) st = prompt_map(&mv, v, bf16, d, 0, a.heads, n_k > 0 ? n_k : n_q, v_stride, d == 128 ? 128 : 64);
    if (st != TQ_OK) return st;
    cudaStream_t s = (cudaStream_t)stream;
    return d == 128 ? launch_prompt_128(a, p->part_rows, mq, mk, mv, bf16, s)
                    : launch_prompt_256(a, p->part_rows, mq, mk, mv, bf16, s);
}

tq_status tq_prompt_get_device_error(const tq_prompt* p, uint32_t* flags, void* stream) {
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
