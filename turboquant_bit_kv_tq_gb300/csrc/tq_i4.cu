// The 4-bit cache: handle, store and load.

#include <algorithm>
#include <new>

#include "tq_i4.cuh"

namespace tq {

// ------------------------------------------------------------------- store
// One vector per group of d/16 lanes; a lane has the 16 elements of one scale.
// The vector's exponent comes from the maximum over its lanes; the rest is the lane's own.
// A block takes consecutive tokens of one KV head, whose rows lie side by side in a page;
// neighbouring blocks take the other heads of the same tokens.  Bound by memory (2 or 4
// bytes in and 4.56 bits out per element), with the instructions close behind (80% of
// the issue slots): 65536 tokens x 8 heads, d = 128, bf16: 59 us, 5860 GB/s (86% of a
// plain copy).
struct I4StoreArgs {
    const void *k, *v;
    int64_t k_stride, v_stride, n_tokens;  // strides in elements
    const int64_t* slots;
    uint8_t* cache;
    int64_t num_slots;
    int heads;
    bool wide;  // rows start at multiples of 32 bytes
    uint32_t* err;
};

constexpr int kI4StoreThreads = 128;

// 32 bytes at once: a whole sector of memory
__device__ __forceinline__ void i4_load32(const uint4* p, uint4& a, uint4& b) {
    // (volatile: it stays behind the wait for the previous kernel)
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void i4_store32(uint4* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// 16 elements, as they lie in memory
template <int DT>
struct I4Raw {
    static constexpr int N = DT == TQ_DTYPE_F32 ? 4 : 2;
    uint4 w[N];
    __device__ __forceinline__ void load(const void* base, int64_t off, bool wide) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + off * (DT == TQ_DTYPE_F32 ? 4 : 2));
        if (wide) {
#pragma unroll
            for (int i = 0; i < N; i += 2) i4_load32(p + i, w[i], w[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __ldg(p + i);
        }
    }
    // the largest magnitude's fp32 bits: without the sign a number's bits are ordered
    // like integers, inf and NaN above every number
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = 0;
        if constexpr (DT == TQ_DTYPE_F32) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                m = max(max(m, max(w[i].x & 0x7FFFFFFFu, w[i].y & 0x7FFFFFFFu)),
                        max(w[i].z & 0x7FFFFFFFu, w[i].w & 0x7FFFFFFFu));
            return m;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                m = __vmaxu2(__vmaxu2(m, __vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu)),
                             __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu));
            const float2 f = DT == TQ_DTYPE_BF16 ? F8Elem::from_bf16x2(m) : F8Elem::from_f16x2(m);
            return max(__float_as_uint(f.x), __float_as_uint(f.y));
        }
    }
    __device__ __forceinline__ float value(int i) const {
        const uint4 q = w[DT == TQ_DTYPE_F32 ? i >> 2 : i >> 3];
        const int j = DT == TQ_DTYPE_F32 ? i & 3 : (i & 7) >> 1;
        const uint32_t u = j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w;
        if constexpr (DT == TQ_DTYPE_F32) return __uint_as_float(u);
        const float2 f = DT == TQ_DTYPE_BF16 ? F8Elem::from_bf16x2(u) : F8Elem::from_f16x2(u);
        return i & 1 ? f.y : f.x;
    }
};

// Codes, scale byte and exponent byte of a lane's 16 elements; `mine` and `top` are
// the fp32 bits of the largest magnitudes among them and in the vector.
//
// Rounding is by addition: q + 1.5 * 2^23 has the integer next to q (ties to even) in
// its low bits, so no conversion is needed, and eight sums times powers of 16 add up to
// a word of codes.  16-bit elements and scales of four bits leave quotients that are
// a tie or 2^-13.9 and more away from one.  So q = x / s is first rounded to a multiple
// of 2^-14, by a sum with 768: that makes a tie of what the rounded reciprocal left next
// to one, and moves nothing across one.  The largest of a group may be 7.5 s, which has
// to go to 7: then the reciprocal is taken 4.37e-6 smaller, which is half of 2^-14 and
// more at 7.5 but less at 6.5 and below.  (All significands, scales and shifts were
// tried.)  With rounding and clamping instructions, which run at a quarter and half of
// the rate, 65536 tokens x 8 heads took 82 us.
constexpr float kI4Round = 12582912.f;  // 1.5 * 2^23 = 0x4B400000
constexpr uint32_t kI4Bias = 0x88888888u - 0x11111111u * 0x4B400000u;

template <int DT>
__device__ __forceinline__ uint2 i4_encode16(const I4Raw<DT>& raw, uint32_t mine, uint32_t top, uint32_t& u, uint32_t& ebyte) {
    const bool bad = top >= 0x7F800000u;
    // smallest E >= 1 with top <= 240 * 2^(E - 127) = 1.875 * 2^(E - 120); at most 248
    const int e = max((int)((top + 0x0FFFFFu) >> 23) - 7, 1);
    ebyte = bad ? 255u : (uint32_t)e;
    const float inv = __uint_as_float((uint32_t)(254 - min(e, 254)) << 23);  // 2^(127 - E)
    const float g = bad ? 0.f : __uint_as_float(mine) * inv;
    // the scale byte: the fp16 number cut off below g / 7.5, whose rounding moves it by
    // less than a step, and then up until 7.5 S(u) (8 bits: exact) reaches g
    u = max((uint32_t)__half_as_ushort(__float2half_rz(g * (2.f / 15.f))) >> 7, 1u);
    u += 7.5f * i4_scale(u) < g;
    u += 7.5f * i4_scale(u) < g;
    if (g <= 0x1p-18f) u = 0;
    const float s = i4_scale(u);
    float r = u ? __frcp_rn(s) : 0.f;
    uint32_t c[2] = {kI4Bias, kI4Bias};
    if constexpr (DT == TQ_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float y = raw.value(i) * inv;
            // The quotient y / s: a product with the rounded reciprocal and one correction,
            // y - q s being exact, so that a tie comes out as one.  24 bits come so near
            // to a tie that the quotient rounds to it: the exact remainder decides
            float q = y * r;
            q = fmaf(fmaf(-q, s, y), r, q);
            float n = (q + kI4Round) - kI4Round;
            const float rest = fmaf(-n, s, y), half = 0.5f * s;
            n += rest > half ? 1.f : rest < -half ? -1.f : 0.f;
            n = u ? fminf(fmaxf(n, -7.f), 7.f) : 0.f;
            c[i / 8] += __float_as_uint(n + kI4Round) << (4 * (i & 7));
        }
    } else {
        if (g == 7.5f * s) r *= 1.f - 4.37e-6f;
        auto codes = [&](float r, auto value) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float q = fmaf(value(i), r, 768.f);
                c[i / 8] += __float_as_uint(q + (kI4Round - 768.f)) * (1u << (4 * (i & 7)));
            }
        };
        // 2^(127 - E) goes into the reciprocal, where that stays in range
        if (!__any_sync(0xffffffffu, e < 40)) codes(r * inv, [&](int i) { return raw.value(i); });
        else codes(r, [&](int i) { return raw.value(i) * inv; });
    }
    return bad ? make_uint2(0x88888888u, 0x88888888u) : make_uint2(c[0], c[1]);
}

template <int D, int DT>
__global__ void __launch_bounds__(kI4StoreThreads) i4_store_kernel(I4StoreArgs a) {
    constexpr int LPV = D / 16;  // lanes per vector
    constexpr int PAGE = i4_page_bytes(D);
    const int sub = threadIdx.x % LPV;
    const int group = blockIdx.x / (unsigned)a.heads, h = blockIdx.x - (unsigned)group * a.heads;
    const int64_t t = (int64_t)group * (kI4StoreThreads / LPV) + threadIdx.x / LPV;
    pdl_wait();  // (the launch overlaps the previous kernel's end)
    // whole warps stay for the shuffles; lanes of a vector share every decision
    I4Raw<DT> k = {}, v = {};
    int64_t slot = -1;
    if (t < a.n_tokens) {
        slot = __ldg(a.slots + t);
        k.load(a.k, t * a.k_stride + (int64_t)h * D + 16 * sub, a.wide);
        v.load(a.v, t * a.v_stride + (int64_t)h * D + 16 * sub, a.wide);
    }
    if (slot >= a.num_slots || slot < -1) {
        if (sub == 0) set_error(a.err, TQ_DEVERR_SLOT);
        slot = -1;
    }
    const uint32_t mk = k.top(), mv = v.top();
    uint32_t tk = mk, tv = mv;
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1) {
        tk = max(tk, __shfl_xor_sync(0xffffffffu, tk, o));
        tv = max(tv, __shfl_xor_sync(0xffffffffu, tv, o));
    }
    uint32_t uk, uv, ek, ev;
    const uint2 ck = i4_encode16<DT>(k, mk, tk, uk, ek), cv = i4_encode16<DT>(v, mv, tv, uv, ev);
    if (slot < 0) return;
    uint8_t* page = a.cache + ((slot >> 4) * a.heads + h) * PAGE;
    const int row = (int)(slot & 15);
    *reinterpret_cast<uint2*>(page + row * (D / 2) + 8 * sub) = ck;
    *reinterpret_cast<uint2*>(page + 8 * D + row * (D / 2) + 8 * sub) = cv;
    page[i4_scales_at(D) + row * LPV + sub] = (uint8_t)uk;
    page[i4_scales_at(D) + D + row * LPV + sub] = (uint8_t)uv;
    if (sub == 0) {
        page[i4_exps_at(D) + row] = (uint8_t)ek;
        page[i4_exps_at(D) + 16 + row] = (uint8_t)ev;
    }
}

template <int D, int DT>
static tq_status launch_i4_store(const I4StoreArgs& a, cudaStream_t s) {
    constexpr int VPB = kI4StoreThreads / (D / 16);
    const int64_t groups = (a.n_tokens + VPB - 1) / VPB;
    if (groups > 0x7FFFFFFF / a.heads) return TQ_ERR_INVALID_ARG;
    return cuda_status(launch_pdl(true, i4_store_kernel<D, DT>, dim3((unsigned)(groups * a.heads)), dim3(kI4StoreThreads), 0, s, a));
}

// -------------------------------------------------------------------- load
// The pages of all sequences, in the order (sequence, page, KV head), are dealt out to
// the warps of a fixed grid; a warp reads one page and writes its 16 rows of keys and
// of values, a lane 16 elements (one scale) at a time.  Bound by memory, four fifths of it
// writes: 16 sequences of up to 16384 tokens, 8 heads, d = 128, to bf16: 110 us, 6430 GB/s
// (95% of a plain copy); with 16-byte stores, half a sector each, 129.  (Sequence by sequence
// the walk alone took every warp a quarter of a microsecond each: 100 x up to 700 53 us, now 33.)
struct I4LoadArgs {
    const uint8_t* cache;
    const int32_t *table, *lens, *cu;
    int batch, heads, max_blocks;
    int64_t num_blocks, n_rows;
    void *k, *v;
    bool wide;  // rows start at multiples of 32 bytes
    uint32_t* err;
};

constexpr int kI4LoadThreads = 256;

template <int OT>
__device__ __forceinline__ void i4_put16(void* base, int64_t off, uint2 codes, float scale, bool wide) {
    float f[16];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = __half22float2(i4_pair(j ? codes.y : codes.x, i));
            f[8 * j + i] = x.x * scale, f[8 * j + 4 + i] = x.y * scale;
        }
    if (!wide) {
        f8_store16(base, off, f, OT);
        return;
    }
    uint4 w[OT == TQ_DTYPE_F32 ? 4 : 2];
    if constexpr (OT == TQ_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                              __float_as_uint(f[4 * i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = make_uint4(f8_pack16(f[8 * i], f[8 * i + 1], OT), f8_pack16(f[8 * i + 2], f[8 * i + 3], OT),
                              f8_pack16(f[8 * i + 4], f[8 * i + 5], OT), f8_pack16(f[8 * i + 6], f[8 * i + 7], OT));
    }
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + off * (OT == TQ_DTYPE_F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (OT == TQ_DTYPE_F32 ? 4 : 2); i += 2) i4_store32(p + i, w[i], w[i + 1]);
}

template <int D, int OT>
__global__ void __launch_bounds__(kI4LoadThreads) i4_load_kernel(I4LoadArgs a) {
    constexpr int PAGE = i4_page_bytes(D);
    constexpr int CPR = D / 16;  // pieces of a row
    const int lane = threadIdx.x & 31;
    const uint32_t warps = gridDim.x * (kI4LoadThreads / 32);
    const uint32_t w0 = blockIdx.x * (kI4LoadThreads / 32) + (threadIdx.x >> 5);
    const int cap = a.max_blocks * 16;
    pdl_wait();  // (the launch overlaps the previous kernel's end)
    // the walk over the sequences, 32 at a time, is the same for every warp: warp w takes
    // the units w, w + warps, ... of the running count (which the configuration keeps in 32 bits)
    uint32_t done = 0;  // units before sequence b0
    uint32_t next = w0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int bl = b0 + lane;
        int len = bl < a.batch ? __ldg(a.lens + bl) : 0;
        if (len < 0 || len > cap) {
            if (w0 == 0) set_error(a.err, TQ_DEVERR_SEQLEN);
            len = len < 0 ? 0 : cap;
        }
        const int start = bl < a.batch ? __ldg(a.cu + bl) : 0;
        const uint32_t mine = (uint32_t)((len + 15) >> 4) * (uint32_t)a.heads;
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
        while (next - done < all) {
            const uint32_t at = next - done;
            next += warps;
            const int i = __ffs(__ballot_sync(0xffffffffu, at < incl)) - 1;  // its sequence
            const int n = __shfl_sync(0xffffffffu, len, i);
            const int row0 = __shfl_sync(0xffffffffu, start, i);
            const uint32_t u = at - __shfl_sync(0xffffffffu, incl - mine, i);
            const int p = (int)(u / (uint32_t)a.heads), h = (int)(u - (uint32_t)p * (uint32_t)a.heads);
            const int blk = __ldg(a.table + (int64_t)(b0 + i) * a.max_blocks + p);
            if (blk < 0 || blk >= a.num_blocks) {
                if (lane == 0) set_error(a.err, TQ_DEVERR_BLOCK);
                continue;
            }
            const uint8_t* page = a.cache + ((int64_t)blk * a.heads + h) * PAGE;
            const int rows = min(16, n - 16 * p);
            const uint32_t eb = __ldg(page + i4_exps_at(D) + lane);  // lanes 0-15: keys, 16-31: values
            uint2 c[CPR];
            uint32_t sb[CPR];
#pragma unroll
            for (int j = 0; j < CPR; ++j) {
                c[j] = __ldg(reinterpret_cast<const uint2*>(page) + lane + 32 * j);
                sb[j] = __ldg(page + i4_scales_at(D) + lane + 32 * j);
            }
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
                // (exact: multiples of 2^-144, at most 2^127)
                i4_put16<OT>(r < 16 ? a.k : a.v, (row * a.heads + h) * D + 16 * ch, c[j], i4_scale(sb[j]) * scale, a.wide);
            }
        }
        done += all;
    }
}

template <int D, int OT>
static tq_status launch_i4_load(const I4LoadArgs& a, cudaStream_t s) {
    int sms = 0;
    const tq_status st = device_sms(&sms);
    if (st != TQ_OK) return st;
    // pages there may be: those of the table, and of the rows to be written.  Two of them a warp,
    // from 8 to 32 blocks per SM: blocks that follow one another keep to fewer places in memory
    // (16 x up to 16384: 8 per SM 115.8 us, 16 112, 24 110, 32 108.4; 100 x up to 700: 8 to 16 33,
    // 32 35)
    const int64_t most = std::min((int64_t)a.batch * a.max_blocks, (a.n_rows >> 4) + a.batch) * a.heads;
    constexpr int W = kI4LoadThreads / 32;
    const int64_t blocks = std::min((most + W - 1) / W, std::max((int64_t)sms * 8, std::min((int64_t)sms * 32, most / (2 * W))));
    return cuda_status(launch_pdl(true, i4_load_kernel<D, OT>, dim3((unsigned)blocks), dim3(kI4LoadThreads), 0, s, a));
}

static bool i4_dtype_ok(int t) { return t == TQ_DTYPE_F32 || t == TQ_DTYPE_BF16 || t == TQ_DTYPE_F16; }
static int i4_dtype_bytes(int t) { return t == TQ_DTYPE_F32 ? 4 : 2; }

static tq_status i4_check(const tq_i4_config& c) {
    if (c.head_dim != 128 && c.head_dim != 256) return TQ_ERR_UNSUPPORTED;
    if (c.block_size != kBlock) return TQ_ERR_UNSUPPORTED;
    if (c.num_kv_heads < 1 || c.num_q_heads < c.num_kv_heads || c.num_q_heads % c.num_kv_heads) return TQ_ERR_INVALID_ARG;
    if (c.num_blocks < 1 || c.num_blocks > 0x7FFFFFFF || c.max_batch < 1 || c.max_blocks_per_seq < 1 ||
        c.max_blocks_per_seq > 0x7FFFFFFF / kBlock)
        return TQ_ERR_INVALID_ARG;
    // q rows and the pages of all block-table entries, KV heads and head groups within int32
    const int nhg = paged_geom(c).nhg;
    if ((int64_t)c.max_batch * c.num_q_heads > 0x7FFFFFFF ||
        (double)c.max_batch * (c.max_blocks_per_seq + paged_unit_cost(4)) * c.num_kv_heads * nhg > 2147483647.0 ||
        (double)c.num_blocks * c.num_kv_heads > 2147483647.0)
        return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_i4_cache_sizes(const tq_i4_config* cfg, size_t* page_bytes, size_t* cache_bytes,
                            size_t* workspace_bytes) {
    if (!cfg) return TQ_ERR_INVALID_ARG;
    const tq_status st = i4_check(*cfg);
    if (st != TQ_OK) return st;
    const size_t page = i4_page_bytes(cfg->head_dim);
    if (page_bytes) *page_bytes = page;
    if (cache_bytes) *cache_bytes = (size_t)cfg->num_blocks * cfg->num_kv_heads * page;
    if (workspace_bytes) *workspace_bytes = paged_workspace(*cfg).total;
    return TQ_OK;
}

tq_status tq_i4_cache_create(const tq_i4_config* cfg, void* workspace_dev, void* stream, tq_i4_cache** out) {
    if (!cfg || !workspace_dev || !out) return TQ_ERR_INVALID_ARG;
    *out = nullptr;
    const tq_status st = i4_check(*cfg);
    if (st != TQ_OK) return st;
    if ((uintptr_t)workspace_dev & 15) return TQ_ERR_MISALIGNED;
    tq_i4_cache* h = new (std::nothrow) tq_i4_cache();
    if (!h) return TQ_ERR_INVALID_ARG;
    const PagedWorkspace w = paged_workspace(*cfg);
    uint8_t* ws = static_cast<uint8_t*>(workspace_dev);
    h->cfg = *cfg;
    h->geom = paged_geom(*cfg);
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

tq_status tq_i4_cache_destroy(tq_i4_cache* cache) {
    delete cache;
    return TQ_OK;
}

tq_status tq_i4_store(const tq_i4_cache* c, const void* k, const void* v, int in_dtype, int64_t k_stride,
                      int64_t v_stride, int64_t num_tokens, const int64_t* slot_mapping, void* cache_buf,
                      void* stream) {
    if (!c || num_tokens < 0) return TQ_ERR_INVALID_ARG;
    if (num_tokens == 0) return TQ_OK;
    if (!k || !v || !slot_mapping || !cache_buf || !i4_dtype_ok(in_dtype)) return TQ_ERR_INVALID_ARG;
    const int64_t row = (int64_t)c->cfg.num_kv_heads * c->cfg.head_dim;
    if (k_stride < row || v_stride < row) return TQ_ERR_INVALID_ARG;
    const int sz = i4_dtype_bytes(in_dtype);
    if ((((uintptr_t)k | (uintptr_t)v | (uintptr_t)(k_stride * sz) | (uintptr_t)(v_stride * sz)) & 15) ||
        ((uintptr_t)cache_buf & 15) || ((uintptr_t)slot_mapping & 7))
        return TQ_ERR_MISALIGNED;
    I4StoreArgs a;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.n_tokens = num_tokens;
    a.slots = slot_mapping;
    a.cache = static_cast<uint8_t*>(cache_buf);
    a.num_slots = c->cfg.num_blocks * kBlock;
    a.heads = c->cfg.num_kv_heads;
    a.wide = !(((uintptr_t)k | (uintptr_t)v | (uintptr_t)(k_stride * sz) | (uintptr_t)(v_stride * sz)) & 31);
    a.err = c->err;
    cudaStream_t s = (cudaStream_t)stream;
    if (c->cfg.head_dim == 128)
        return in_dtype == TQ_DTYPE_F32    ? launch_i4_store<128, TQ_DTYPE_F32>(a, s)
               : in_dtype == TQ_DTYPE_BF16 ? launch_i4_store<128, TQ_DTYPE_BF16>(a, s)
                                           : launch_i4_store<128, TQ_DTYPE_F16>(a, s);
    return in_dtype == TQ_DTYPE_F32    ? launch_i4_store<256, TQ_DTYPE_F32>(a, s)
           : in_dtype == TQ_DTYPE_BF16 ? launch_i4_store<256, TQ_DTYPE_BF16>(a, s)
                                       : launch_i4_store<256, TQ_DTYPE_F16>(a, s);
}

tq_status tq_i4_load(const tq_i4_cache* c, const void* cache_buf, const int32_t* block_table,
                     const int32_t* seq_lens, const int32_t* cu_out, int batch, int64_t n_rows, void* k_out,
                     void* v_out, int out_dtype, void* stream) {
    if (!c || !cache_buf || !block_table || !seq_lens || !cu_out || n_rows < 0) return TQ_ERR_INVALID_ARG;
    if (batch < 1 || batch > c->cfg.max_batch || !i4_dtype_ok(out_dtype)) return TQ_ERR_INVALID_ARG;
    if (n_rows > 0 && (!k_out || !v_out)) return TQ_ERR_INVALID_ARG;
    if (((uintptr_t)cache_buf | (uintptr_t)k_out | (uintptr_t)v_out) & 15) return TQ_ERR_MISALIGNED;
    I4LoadArgs a;
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
    a.wide = !(((uintptr_t)k_out | (uintptr_t)v_out) & 31);
    a.err = c->err;
    cudaStream_t s = (cudaStream_t)stream;
    if (c->cfg.head_dim == 128)
        return out_dtype == TQ_DTYPE_F32    ? launch_i4_load<128, TQ_DTYPE_F32>(a, s)
               : out_dtype == TQ_DTYPE_BF16 ? launch_i4_load<128, TQ_DTYPE_BF16>(a, s)
                                            : launch_i4_load<128, TQ_DTYPE_F16>(a, s);
    return out_dtype == TQ_DTYPE_F32    ? launch_i4_load<256, TQ_DTYPE_F32>(a, s)
           : out_dtype == TQ_DTYPE_BF16 ? launch_i4_load<256, TQ_DTYPE_BF16>(a, s)
                                        : launch_i4_load<256, TQ_DTYPE_F16>(a, s);
}

tq_status tq_i4_get_device_error(const tq_i4_cache* c, uint32_t* flags, void* stream) {
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
