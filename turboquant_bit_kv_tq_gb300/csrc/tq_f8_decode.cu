// Decode attention over the 8-bit cache.

#include "tq_paged_decode.cuh"

extern "C" tq_status tq_f8_decode_attention(const tq_f8_cache* c, const void* q, int q_dtype, int64_t q_stride,
                                            const void* cache_buf, const int32_t* block_table,
                                            const int32_t* seq_lens, float scale, int batch, void* out,
                                            int out_dtype, void* stream) {
    return tq::paged_decode<8>(c, q, q_dtype, q_stride, cache_buf, block_table, seq_lens, scale, batch, out, out_dtype,
                               stream);
}
