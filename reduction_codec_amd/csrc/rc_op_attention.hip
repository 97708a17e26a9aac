// Attention over a paged cache in MXFP4: the workspace and the type's kernels.
#include "rc_op_attention.hpp"

namespace rc {

hipError_t launch_attention_bf16(int d, const CacheAttention& a, size_t rows, hipStream_t st);
hipError_t launch_attention_fp16(int d, const CacheAttention& a, size_t rows, hipStream_t st);
hipError_t launch_attention_fp32(int d, const CacheAttention& a, size_t rows, hipStream_t st);

// By sizes alone: the most that any type of queries takes.
size_t cache_attention_work(size_t tokens, size_t heads, size_t kv_heads, size_t d)
{
    const size_t rows = tokens > 0x7FFFFFFF ? tokens : tokens * (heads / kv_heads);
    const size_t b = attention_work_t<kBF16>((int)d, rows, kv_heads), h = attention_work_t<kF16>((int)d, rows, kv_heads), f = attention_work_t<kF32>((int)d, rows, kv_heads);
    return b > h ? (b > f ? b : f) : h > f ? h : f;
}

hipError_t launch_cache_attention(int dt, int d, const CacheAttention& a, size_t max_query, hipStream_t st)
{
    const size_t tokens = a.c.tokens, most = max_query != 0 && max_query < tokens ? max_query : tokens;
    const size_t rows = most * (a.heads / a.c.kv_heads);
    return dt == kF32 ? launch_attention_fp32(d, a, rows, st) : dt == kF16 ? launch_attention_fp16(d, a, rows, st)
                                                                         : launch_attention_bf16(d, a, rows, st);
}

}  // namespace rc
