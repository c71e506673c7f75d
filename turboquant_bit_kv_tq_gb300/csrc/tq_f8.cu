// The 8-bit cache: handle, store and load.

#include <algorithm>
#include <new>

#include "tq_f8.cuh"

namespace tq {

// ------------------------------------------------------------------- store
// One vector per group of d/8 lanes, 8 elements per lane.  Maximum over the
// lanes, exact scaling by a power of two, one conversion to e4m3.  Bound by
// memory: 2 (or 4) bytes in and 1 out per element.  A block takes consecutive
// tokens of one KV head, whose rows lie side by side in a page; neighbouring
// blocks take the other heads of the same tokens.  The vectors are loaded before
// their slot is known, so that a block waits for memory once.  65536 tokens x 8 heads,
// d = 128, bf16: 64 us, 6290 GB/s (93% of a plain copy's 6786); with the slot
// loaded first and a block's warps on different heads it took 77.
struct F8StoreArgs {
    const void *k, *v;
    int64_t k_stride, v_stride, n_tokens;  // strides in elements
    const int64_t* slots;
    uint8_t* cache;
    int64_t num_slots;
    int heads;
    uint32_t* err;
};

constexpr int kF8StoreThreads = 128;

// 8 elements, as they lie in memory
template <int DT>
struct F8Raw {
    uint4 w[DT == TQ_DTYPE_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, int64_t off) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + off * (DT == TQ_DTYPE_F32 ? 4 : 2));
        w[0] = __ldg(p);
        if constexpr (DT == TQ_DTYPE_F32) w[1] = __ldg(p + 1);
    }
    // largest magnitude: as a number's bits without the sign they are ordered like
    // integers, inf and NaN above every number.  16-bit types: two maxima, packed
    __device__ __forceinline__ uint32_t top() const {
        if constexpr (DT == TQ_DTYPE_F32) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                m = max(max(m, max(w[i].x & 0x7FFFFFFFu, w[i].y & 0x7FFFFFFFu)),
                        max(w[i].z & 0x7FFFFFFFu, w[i].w & 0x7FFFFFFFu));
            return m;
        } else {
            return __vmaxu2(__vmaxu2(w[0].x & 0x7FFF7FFFu, w[0].y & 0x7FFF7FFFu),
                            __vmaxu2(w[0].z & 0x7FFF7FFFu, w[0].w & 0x7FFF7FFFu));
        }
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[DT == TQ_DTYPE_F32].x, w[DT == TQ_DTYPE_F32].y,
                               w[DT == TQ_DTYPE_F32].z, w[DT == TQ_DTYPE_F32].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (DT == TQ_DTYPE_F32) {
                x[i] = __uint_as_float(u[i]);
            } else {
                const float2 f = DT == TQ_DTYPE_BF16 ? F8Elem::from_bf16x2(u[i >> 1]) : F8Elem::from_f16x2(u[i >> 1]);
                x[i] = i & 1 ? f.y : f.x;
            }
        }
    }
};

// codes and exponent byte of 8 elements, from the vector's largest magnitude (fp32 bits)
template <int DT>
__device__ __forceinline__ uint2 f8_encode8(const F8Raw<DT>& raw, uint32_t top, uint32_t& ebyte) {
    const bool bad = top >= 0x7F800000u;
    // smallest e with top <= 448 * 2^e = 1.75 * 2^(e + 8); at most 120, so no upper clamp
    const int e = max((int)((top + 0x1FFFFFu) >> 23) - 8, 1);
    ebyte = bad ? 255u : (uint32_t)e;
    const float inv = __uint_as_float((uint32_t)(254 - min(e, 254)) << 23);  // 2^(127 - e)
    float x[8];
    raw.values(x);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x[2 * i + 1] * inv), "f"(x[2 * i] * inv));
        c[i] = r;
    }
    return bad ? make_uint2(0u, 0u) : make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int D, int DT>
__global__ void __launch_bounds__(kF8StoreThreads) f8_store_kernel(F8StoreArgs a) {
    constexpr int LPV = D / 8;  // lanes per vector
    constexpr int PAGE = f8_page_bytes(D);
    const int sub = threadIdx.x % LPV;
    const int group = blockIdx.x / (unsigned)a.heads, h = blockIdx.x - (unsigned)group * a.heads;
    const int64_t t = (int64_t)group * (kF8StoreThreads / LPV) + threadIdx.x / LPV;
    pdl_wait();  // (the launch overlaps the previous kernel's end)
    // whole warps stay for the shuffles; lanes of a vector share every decision
    F8Raw<DT> k = {}, v = {};
    int64_t slot = -1;
    if (t < a.n_tokens) {
        slot = __ldg(a.slots + t);
        k.load(a.k, t * a.k_stride + (int64_t)h * D + 8 * sub);
        v.load(a.v, t * a.v_stride + (int64_t)h * D + 8 * sub);
    }
    if (slot >= a.num_slots || slot < -1) {
        if (sub == 0) set_error(a.err, TQ_DEVERR_SLOT);
        slot = -1;
    }
    uint32_t tk = k.top(), tv = v.top();
    if constexpr (DT == TQ_DTYPE_F32) {
#pragma unroll
        for (int o = LPV / 2; o > 0; o >>= 1) {
            tk = max(tk, __shfl_xor_sync(0xffffffffu, tk, o));
            tv = max(tv, __shfl_xor_sync(0xffffffffu, tv, o));
        }
    } else {
        // both vectors' maxima in one word: one exchange for the two
        uint32_t m = __vmaxu2(__byte_perm(tk, tv, 0x5410), __byte_perm(tk, tv, 0x7632));
#pragma unroll
        for (int o = LPV / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float2 f = DT == TQ_DTYPE_BF16 ? F8Elem::from_bf16x2(m) : F8Elem::from_f16x2(m);
        tk = __float_as_uint(f.x), tv = __float_as_uint(f.y);
    }
    uint32_t ek, ev;
    const uint2 ck = f8_encode8<DT>(k, tk, ek), cv = f8_encode8<DT>(v, tv, ev);
    if (slot < 0) return;
    uint8_t* page = a.cache + ((slot >> 4) * a.heads + h) * PAGE;
    const int row = (int)(slot & 15);
    *reinterpret_cast<uint2*>(page + row * D + 8 * sub) = ck;
    *reinterpret_cast<uint2*>(page + 16 * D + row * D + 8 * sub) = cv;
    if (sub == 0) {
        page[32 * D + row] = (uint8_t)ek;
        page[32 * D + 16 + row] = (uint8_t)ev;
    }
}

template <int D, int DT>
static tq_status launch_f8_store(const F8StoreArgs& a, cudaStream_t s) {
    constexpr int VPB = kF8StoreThreads / (D / 8);
    const int64_t blocks = (a.n_tokens + VPB - 1) / VPB * a.heads;
    if (blocks > 0x7FFFFFFF) return TQ_ERR_INVALID_ARG;
    return cuda_status(launch_pdl(true, f8_store_kernel<D, DT>, dim3((unsigned)blocks), dim3(kF8StoreThreads), 0, s, a));
}

// -------------------------------------------------------------------- load
// The pages of all sequences, in the order (sequence, page, KV head), are
// dealt out to the warps of a fixed grid; a warp reads one page and writes its
// 16 rows of keys and of values.  Bound by memory: 16 sequences of up to 16384 tokens,
// 8 heads, d = 128, to bf16: 133 us, 6230 GB/s (92% of a plain copy).
struct F8LoadArgs {
    const uint8_t* cache;
    const int32_t *table, *lens, *cu;
    int batch, heads, max_blocks;
    int64_t num_blocks, n_rows;
    void *k, *v;
    uint32_t* err;
};

constexpr int kF8LoadThreads = 256;

template <int D, int OT>
__device__ __forceinline__ void f8_put16(void* base, int64_t off, uint4 codes, float scale) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = f8_to_f16x2(w[i]), hi = f8_to_f16x2_hi(w[i]);
        const float2 a = F8Elem::from_f16x2(lo), b = F8Elem::from_f16x2(hi);
        f[4 * i] = a.x * scale, f[4 * i + 1] = a.y * scale, f[4 * i + 2] = b.x * scale, f[4 * i + 3] = b.y * scale;
    }
    if constexpr (OT == TQ_DTYPE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            p[i] = make_uint4(f8_pack16(f[8 * i], f[8 * i + 1], OT), f8_pack16(f[8 * i + 2], f[8 * i + 3], OT),
                              f8_pack16(f[8 * i + 4], f[8 * i + 5], OT), f8_pack16(f[8 * i + 6], f[8 * i + 7], OT));
    }
}

template <int D, int OT>
__global__ void __launch_bounds__(kF8LoadThreads) f8_load_kernel(F8LoadArgs a) {
    constexpr int PAGE = f8_page_bytes(D);
    constexpr int CPR = D / 16;  // 16-byte chunks per row
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kF8LoadThreads / 32);
    const int64_t w0 = (int64_t)blockIdx.x * (kF8LoadThreads / 32) + (threadIdx.x >> 5);
    const int cap = a.max_blocks * 16;
    pdl_wait();  // (the launch overlaps the previous kernel's end)
    // the walk over the sequences is the same for every warp: warp w takes the
    // units w, w + warps, ... of the running count
    int64_t done = 0;  // units before sequence b
    int64_t next = w0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int bl = b0 + lane;
        int len = bl < a.batch ? __ldg(a.lens + bl) : 0;
        if (len < 0 || len > cap) {
            if (w0 == 0) set_error(a.err, TQ_DEVERR_SEQLEN);
            len = len < 0 ? 0 : cap;
        }
        const int start = bl < a.batch ? __ldg(a.cu + bl) : 0;
        const int nb = min(32, a.batch - b0);
        for (int i = 0; i < nb; ++i) {
            const int n = __shfl_sync(0xffffffffu, len, i);
            const int row0 = __shfl_sync(0xffffffffu, start, i);
            const int64_t units = (int64_t)((n + 15) >> 4) * a.heads;
            while (next < done + units) {
                const int64_t u = next - done;
                next += warps;
                const int p = (int)(u / a.heads), h = (int)(u - (int64_t)p * a.heads);
                const int blk = __ldg(a.table + (int64_t)(b0 + i) * a.max_blocks + p);
                if (blk < 0 || blk >= a.num_blocks) {
                    if (lane == 0) set_error(a.err, TQ_DEVERR_BLOCK);
                    continue;
                }
                const uint8_t* page = a.cache + ((int64_t)blk * a.heads + h) * PAGE;
                const int rows = min(16, n - 16 * p);
                const uint32_t eb = __ldg(page + 32 * D + lane);  // lanes 0-15: keys, 16-31: values
                uint4 c[CPR];
#pragma unroll
                for (int j = 0; j < CPR; ++j)
                    c[j] = __ldg(reinterpret_cast<const uint4*>(page) + lane + 32 * j);
#pragma unroll
                for (int j = 0; j < CPR; ++j) {
                    const int idx = lane + 32 * j, r = idx / CPR, ch = idx % CPR;  // r: 0-15 keys, 16-31 values
                    const float scale = f8_scale(__shfl_sync(0xffffffffu, eb, r));
                    const int64_t row = (int64_t)row0 + 16 * p + (r & 15);
                    if ((r & 15) >= rows) continue;
                    if (row < 0 || row >= a.n_rows) {
                        set_error(a.err, TQ_DEVERR_CHUNK);
                        continue;
                    }
                    f8_put16<D, OT>(r < 16 ? a.k : a.v, (row * a.heads + h) * D + 16 * ch, c[j], scale);
                }
            }
            done += units;
        }
    }
}

template <int D, int OT>
static tq_status launch_f8_load(const F8LoadArgs& a, cudaStream_t s) {
    int sms = 0;
    const tq_status st = device_sms(&sms);
    if (st != TQ_OK) return st;
    const int64_t most = (int64_t)a.batch * a.max_blocks * a.heads;
    const int64_t blocks = std::min<int64_t>((most + 7) / 8, (int64_t)sms * 8);
    return cuda_status(launch_pdl(true, f8_load_kernel<D, OT>, dim3((unsigned)blocks), dim3(kF8LoadThreads), 0, s, a));
}

static bool f8_dtype_ok(int t) { return t == TQ_DTYPE_F32 || t == TQ_DTYPE_BF16 || t == TQ_DTYPE_F16; }
static int f8_dtype_bytes(int t) { return t == TQ_DTYPE_F32 ? 4 : 2; }

static tq_status f8_check(const tq_f8_config& c) {
    if (c.head_dim != 128 && c.head_dim != 256) return TQ_ERR_UNSUPPORTED;
    if (c.block_size != kBlock) return TQ_ERR_UNSUPPORTED;
    if (c.num_kv_heads < 1 || c.num_q_heads < c.num_kv_heads || c.num_q_heads % c.num_kv_heads) return TQ_ERR_INVALID_ARG;
    if (c.num_blocks < 1 || c.num_blocks > 0x7FFFFFFF || c.max_batch < 1 || c.max_blocks_per_seq < 1 ||
        c.max_blocks_per_seq > 0x7FFFFFFF / kBlock)
        return TQ_ERR_INVALID_ARG;
    // q rows and the pages of all block-table entries, KV heads and head groups within int32
    const F8Geom g = f8_geom(c);
    if ((int64_t)c.max_batch * c.num_q_heads > 0x7FFFFFFF ||
        (double)c.max_batch * (c.max_blocks_per_seq + kF8UnitCost) * c.num_kv_heads * g.nhg > 2147483647.0 ||
        (double)c.num_blocks * c.num_kv_heads > 2147483647.0)
        return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_f8_cache_sizes(const tq_f8_config* cfg, size_t* page_bytes, size_t* cache_bytes,
                            size_t* workspace_bytes) {
    if (!cfg) return TQ_ERR_INVALID_ARG;
    const tq_status st = f8_check(*cfg);
    if (st != TQ_OK) return st;
    const size_t page = f8_page_bytes(cfg->head_dim);
    if (page_bytes) *page_bytes = page;
    if (cache_bytes) *cache_bytes = (size_t)cfg->num_blocks * cfg->num_kv_heads * page;
    if (workspace_bytes) *workspace_bytes = f8_workspace(*cfg).total;
    return TQ_OK;
}

tq_status tq_f8_cache_create(const tq_f8_config* cfg, void* workspace_dev, void* stream, tq_f8_cache** out) {
    if (!cfg || !workspace_dev || !out) return TQ_ERR_INVALID_ARG;
    *out = nullptr;
    const tq_status st = f8_check(*cfg);
    if (st != TQ_OK) return st;
    if ((uintptr_t)workspace_dev & 15) return TQ_ERR_MISALIGNED;
    tq_f8_cache* h = new (std::nothrow) tq_f8_cache();
    if (!h) return TQ_ERR_INVALID_ARG;
    const F8Workspace w = f8_workspace(*cfg);
    uint8_t* ws = static_cast<uint8_t*>(workspace_dev);
    h->cfg = *cfg;
    h->geom = f8_geom(*cfg);
    h->err = reinterpret_cast<uint32_t*>(ws + w.err);
    h->cnt = reinterpret_cast<uint32_t*>(ws + w.cnt);
    h->gcnt = reinterpret_cast<uint32_t*>(ws + w.gcnt);
    h->part = reinterpret_cast<float4*>(ws + w.part);
    h->meta = reinterpret_cast<float4*>(ws + w.meta);
    cudaStream_t s = (cudaStream_t)stream;
    tq_status cs = cuda_status(cudaMemsetAsync(ws, 0, w.zeroed, s));
    if (cs == TQ_OK) cs = cuda_status(cudaStreamSynchronize(s));
    if (cs != TQ_OK) {
        delete h;
        return cs;
    }
    *out = h;
    return TQ_OK;
}

tq_status tq_f8_cache_destroy(tq_f8_cache* cache) {
    delete cache;
    return TQ_OK;
}

tq_status tq_f8_store(const tq_f8_cache* c, const void* k, const void* v, int in_dtype, int64_t k_stride,
                      int64_t v_stride, int64_t num_tokens, const int64_t* slot_mapping, void* cache_buf,
                      void* stream) {
    if (!c || num_tokens < 0) return TQ_ERR_INVALID_ARG;
    if (num_tokens == 0) return TQ_OK;
    if (!k || !v || !slot_mapping || !cache_buf || !f8_dtype_ok(in_dtype)) return TQ_ERR_INVALID_ARG;
    const int64_t row = (int64_t)c->cfg.num_kv_heads * c->cfg.head_dim;
    if (k_stride < row || v_stride < row) return TQ_ERR_INVALID_ARG;
    const int sz = f8_dtype_bytes(in_dtype);
    if ((((uintptr_t)k | (uintptr_t)v | (uintptr_t)(k_stride * sz) | (uintptr_t)(v_stride * sz)) & 15) ||
        ((uintptr_t)cache_buf & 15) || ((uintptr_t)slot_mapping & 7))
        return TQ_ERR_MISALIGNED;
    F8StoreArgs a;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.n_tokens = num_tokens;
    a.slots = slot_mapping;
    a.cache = static_cast<uint8_t*>(cache_buf);
    a.num_slots = c->cfg.num_blocks * kBlock;
    a.heads = c->cfg.num_kv_heads;
    a.err = c->err;
    cudaStream_t s = (cudaStream_t)stream;
    if (c->cfg.head_dim == 128)
        return in_dtype == TQ_DTYPE_F32    ? launch_f8_store<128, TQ_DTYPE_F32>(a, s)
               : in_dtype == TQ_DTYPE_BF16 ? launch_f8_store<128, TQ_DTYPE_BF16>(a, s)
                                           : launch_f8_store<128, TQ_DTYPE_F16>(a, s);
    return in_dtype == TQ_DTYPE_F32    ? launch_f8_store<256, TQ_DTYPE_F32>(a, s)
           : in_dtype == TQ_DTYPE_BF16 ? launch_f8_store<256, TQ_DTYPE_BF16>(a, s)
                                       : launch_f8_store<256, TQ_DTYPE_F16>(a, s);
}

tq_status tq_f8_load(const tq_f8_cache* c, const void* cache_buf, const int32_t* block_table,
                     const int32_t* seq_lens, const int32_t* cu_out, int batch, int64_t n_rows, void* k_out,
                     void* v_out, int out_dtype, void* stream) {
    if (!c || !cache_buf || !block_table || !seq_lens || !cu_out || n_rows < 0) return TQ_ERR_INVALID_ARG;
    if (batch < 1 || batch > c->cfg.max_batch || !f8_dtype_ok(out_dtype)) return TQ_ERR_INVALID_ARG;
    if (n_rows > 0 && (!k_out || !v_out)) return TQ_ERR_INVALID_ARG;
    if (((uintptr_t)cache_buf | (uintptr_t)k_out | (uintptr_t)v_out) & 15) return TQ_ERR_MISALIGNED;
    F8LoadArgs a;
    a.cache = static_cast<const uint8_t*>(cache_buf);
    a.table = block_table;
    a.lens = seq_lens;
    a.cu = cu_out;
    a.batch = batch;
    a.heads = c->cfg.num_kv_heads;
    a.max_blocks = c->cfg.max_blocks_per_seq;
    a.num_blocks = c->cfg.num_blocks;
    a.n_rows = n_rows;
    a.k = k_out;
    a.v = v_out;
    a.err = c->err;
    cudaStream_t s = (cudaStream_t)stream;
    if (c->cfg.head_dim == 128)
        return out_dtype == TQ_DTYPE_F32    ? launch_f8_load<128, TQ_DTYPE_F32>(a, s)
               : out_dtype == TQ_DTYPE_BF16 ? launch_f8_load<128, TQ_DTYPE_BF16>(a, s)
                                            : launch_f8_load<128, TQ_DTYPE_F16>(a, s);
    return out_dtype == TQ_DTYPE_F32    ? launch_f8_load<256, TQ_DTYPE_F32>(a, s)
           : out_dtype == TQ_DTYPE_BF16 ? launch_f8_load<256, TQ_DTYPE_BF16>(a, s)
                                        : launch_f8_load<256, TQ_DTYPE_F16>(a, s);
}

tq_status tq_f8_get_device_error(const tq_f8_cache* c, uint32_t* flags, void* stream) {
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
