// e0_attn_decode (the kernels: e0_attn.cuh).
#include "e0_attn.cuh"

namespace e0 {

size_t attn_ws_bytes(int D) {
    const size_t slots = 2 * (size_t)attn_blocks();
    return slots * MOST_ROWS * D * sizeof(float) + slots * MOST_ROWS * sizeof(float2) + slots * sizeof(Cut);
}

int attn_decode(const e0_kv_cache* c, const int32_t* table, int max_blocks, const int32_t* ctx, const int32_t* cu,
                int B, int max_q, const void* q, int dtype, int64_t q_ld, int Hq, float scale, int window, void* out,
                int64_t out_ld, float* lse, void* ws, uint32_t* st, cudaStream_t s) {
    return launch_t<false>(
        args_of(c, table, max_blocks, ctx, cu, B, max_q, q, q_ld, Hq, scale, window, out, out_ld, lse, ws, st), dtype, c->D, s);
}

}  // namespace e0
