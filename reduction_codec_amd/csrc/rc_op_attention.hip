// Attention over a paged cache held in MXFP4.
//
//   s_j = scale q . K_j,  out = sum exp(s_j - m) V_j / sum exp(s_j - m),
//   lse = m + log sum exp(s_j - m),  m = max s_j
//
// The simplest form: a workgroup has one row of one head and takes its tokens
// 256 at a time, a lane a token for the scores, then a lane a value for the sum.
#include "rc_op_cache.hpp"

namespace rc {
namespace {

constexpr int kT = 256;

__device__ __forceinline__ float value_at(const uint8_t* stream, uint32_t token, uint32_t i, int d)
{
    const uint32_t b = token * (d / 32) + i / 32;
    const uint32_t w = stream[codes_at(b) + i % 32 / 2];
    const f2 p = fp4_dec(w, __uint_as_float((uint32_t)stream[scale_at(b)] << 23), 0);
    return i % 2 ? p.y : p.x;
}

template <int DT>
__global__ __launch_bounds__(kT) void attention_simple_kernel(const CacheAttention a, int d)
{
    __shared__ float q[256], p[kT], slot[kT / 64];
    const int row = blockIdx.x, head = blockIdx.y, t = threadIdx.x;
    const RowPlace at = row_place(a.c, row);
    if (at.seq < 0) return;
    const int kv = head / (a.heads / a.c.kv_heads), mask = (1 << a.c.shift) - 1;
    const int len = seq_length(a.c, at.seq);
    int end = a.causal ? (at.pos + 1 < len ? at.pos + 1 : len) : len;
    int begin = a.window && at.pos - a.window + 1 > 0 ? at.pos - a.window + 1 : 0;
    if (t < d) q[t] = load1<DT>(a.q, (size_t)row * a.q_stride + (size_t)head * d + t);
    float m = -__builtin_inff(), l = 0.0f, o = 0.0f;
    for (int j0 = begin; j0 < end; j0 += kT) {
        __syncthreads();
        const int j = j0 + t;
        float s = -__builtin_inff();
        if (j < end) {
            const int page = page_of(a.c, at.seq, j);
            if (page >= 0) {
                const uint8_t* k = a.c.k + stream_at(a.c, page, kv);
                s = 0.0f;
                for (int i = 0; i < d; ++i) s += q[i] * value_at(k, j & mask, i, d);
                s *= a.scale;
            }
        }
        float top = s;
        for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x, 64));
        if ((t & 63) == 0) slot[t >> 6] = top;
        __syncthreads();
        const float mn = fmaxf(fmaxf(fmaxf(slot[0], slot[1]), fmaxf(slot[2], slot[3])), m);
        const float base = mn == -__builtin_inff() ? 0.0f : mn;
        const float e = expf(s - base), old = expf(m - base);
        p[t] = e;
        m = mn;
        __syncthreads();
        l = l * old;
        o = o * old;
        for (int x = 0; x < kT && j0 + x < end; ++x) {
            l += p[x];
            const int page = page_of(a.c, at.seq, j0 + x);
            if (t < d && page >= 0) o += p[x] * value_at(a.c.v + stream_at(a.c, page, kv), (j0 + x) & mask, t, d);
        }
    }
    const size_t r = (size_t)row * a.heads + head;
    if (t < d) store1<DT>(a.out, r * d + t, l == 0.0f ? 0.0f : o / l);
    if (a.lse && t == 0) a.lse[r] = l == 0.0f ? -__builtin_inff() : m + logf(l);
}

template <int DT>
hipError_t simple(const CacheAttention& a, int d, hipStream_t st)
{
    attention_simple_kernel<DT><<<dim3((unsigned)a.c.tokens, (unsigned)a.heads), kT, 0, st>>>(a, d);
    return hipGetLastError();
}

}  // namespace

size_t cache_attention_work(size_t, size_t, size_t, size_t) { return 16; }

hipError_t launch_cache_attention(int dt, int d, const CacheAttention& a, size_t, hipStream_t st)
{
    return dt == kF32 ? simple<kF32>(a, d, st) : dt == kF16 ? simple<kF16>(a, d, st) : simple<kBF16>(a, d, st);
}

}  // namespace rc
