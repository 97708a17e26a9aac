// Attention over a paged cache in MXFP4: the kernels for bf16 queries.
#include "rc_op_attention.hpp"

namespace rc {

hipError_t launch_attention_bf16(int d, const CacheAttention& a, size_t rows, hipStream_t st)
{
    return attention_t<kBF16>(d, a, rows, st);
}

}  // namespace rc
