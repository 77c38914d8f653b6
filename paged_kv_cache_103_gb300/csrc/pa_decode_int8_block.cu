// pa_decode_int8_block: the decode over a block-scaled cache of INT8 codes.
#include "pa_decode_block8.cuh"

extern "C" {

PA_API pa_status pa_decode_int8_block(const void* q, const void* k_cache, const void* v_cache,
                                      const float* k_scale, const float* v_scale,
                                      const int32_t* block_tables, int32_t max_blocks,
                                      const int32_t* context_lens, int32_t max_context_len,
                                      int32_t B, int32_t H, int32_t Hkv, int32_t d,
                                      int32_t block_size, int32_t num_blocks, float scale,
                                      pa_dtype dtype, void* out, void* workspace,
                                      size_t ws_bytes, void* stream) {
    return decode<true>(q, k_cache, v_cache, k_scale, v_scale, block_tables, max_blocks,
                        context_lens, max_context_len, B, H, Hkv, d, block_size, num_blocks, scale,
                        dtype, out, workspace, ws_bytes, stream);
}

}  // extern "C"
