// Attention over a paged cache in MXFP4: the choice of kernels and the workspace.
#include "rc_op_attention.hpp"

namespace rc {

hipError_t launch_attention_bf16(int d, const CacheAttention& a, size_t most_rows, hipStream_t st);
hipError_t launch_attention_fp16(int d, const CacheAttention& a, size_t most_rows, hipStream_t st);
hipError_t launch_attention_fp32(int d, const CacheAttention& a, size_t most_rows, hipStream_t st);

// By sizes alone, for the type that leaves the largest parts.
size_t cache_attention_work(size_t tokens, size_t heads, size_t kv_heads, size_t d)
{
    const int nb = (int)(d / 32), qt = tokens * (heads / kv_heads) <= 16 ? 1 : 2;
    size_t most = 0;
    for (int q = 1; q <= qt; ++q) {
        const size_t groups = 256 * (size_t)row_groups(1, nb, q);
        const size_t bytes = groups * (sizeof(Cut) + 2 * 16 * q * (d + 2) * sizeof(float));
        most = bytes > most ? bytes : most;
    }
    return most;
}

hipError_t launch_cache_attention(int dt, int d, const CacheAttention& a, size_t max_query, hipStream_t st)
{
    const size_t tokens = a.c.tokens, most = max_query != 0 && max_query < tokens ? max_query : tokens;
    const size_t rows = most * (a.heads / a.c.kv_heads);
    return dt == kF32 ? launch_attention_fp32(d, a, rows, st) : dt == kF16 ? launch_attention_fp16(d, a, rows, st)
                                                                         : launch_attention_bf16(d, a, rows, st);
}

}  // namespace rc
