// Global norm of many tensors, and clipping by it.
//
//   N = |scale| sqrt(sum over all tensors of g^2)
//   out = round(g * scale * min(1, max_norm / (N + eps)))
//
// Two kernels read the tensors through a table in the kernel arguments (no
// device copy of the pointers, so a call can be captured and replayed).  Every
// tensor is cut into 16 KiB chunks; a workgroup walks the chunks of all the
// table's tensors with a stride of the grid and keeps one sum of squares, in
// binary64: the squares of binary32 values neither overflow nor vanish there,
// and the order of the additions, fixed by the sizes alone, does not show in
// the rounded norm.  The second kernel adds the workgroups' sums (each one of
// its workgroups for itself, 16 KiB from L2, which saves a launch and a wait)
// and scales the chunks from the last to the first, so that what the first
// kernel read last is still in the 256 MiB cache.
#include "rc_op.hpp"
#include "rc_op_launch.hpp"

namespace rc {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kChunkBytes = 16384;          // of input: four 16-byte loads per lane
constexpr int kTable = 96;                       // tensors per launch: 96 * 36 bytes of kernel arguments

struct Table {
    const void* in[kTable];
    void* out[kTable];
    uint64_t n[kTable];
    uint64_t first[kTable + 1];                  // first chunk of each tensor, total last
    uint8_t in_t[kTable], out_t[kTable];
    int count;
};

__device__ __forceinline__ uint32_t chunk_elems(int dt) { return kChunkBytes / (dt == kF32 ? 4 : 2); }

__device__ __forceinline__ double wave_total64(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

__device__ __forceinline__ double group_total64(double v, double* slot)
{
    v = wave_total64(v);
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    return (slot[0] + slot[1]) + (slot[2] + slot[3]);
}

// The lane's four vectors of a chunk, +0 beyond the tensor's end.
template <int DT>
__device__ __forceinline__ void load_chunk(const void* in, size_t base, size_t n, u32x4 (&u)[4])
{
    constexpr int E = Elem<DT>::per16, S = Elem<DT>::size;
    const size_t i = base + threadIdx.x * E;
    if (base + chunk_elems(DT) <= n) {           // uniform: all but a tensor's last chunk
#pragma unroll
        for (int j = 0; j < 4; ++j)
            u[j] = *reinterpret_cast<const u32x4_any*>(static_cast<const uint8_t*>(in) + (i + j * kThreads * E) * S);
    } else {
        load_row<DT>(in, i, kThreads * E, n, u);
    }
}

template <int DT>
__device__ __forceinline__ double chunk_squares(const void* in, size_t n, size_t base)
{
    constexpr int E = Elem<DT>::per16;
    u32x4 u[4];
    load_chunk<DT>(in, base, n, u);
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[E];
        widen16<DT>(u[i], v);
#pragma unroll
        for (int e = 0; e < E; ++e) s[e & 1] = fma((double)v[e], (double)v[e], s[e & 1]);
    }
    return s[0] + s[1];
}

// `add`: a later table of the same call adds to the sums of the earlier ones.
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(const Table t, double* partial, int add)
{
    __shared__ double slot[kThreads / 64];
    double s = 0.0;
    int k = 0;
    for (uint64_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        while (c >= t.first[k + 1]) ++k;
        const size_t base = (c - t.first[k]) * chunk_elems(t.in_t[k]);
        s += t.in_t[k] == kF32 ? chunk_squares<kF32>(t.in[k], t.n[k], base)
           : t.in_t[k] == kBF16 ? chunk_squares<kBF16>(t.in[k], t.n[k], base)
                                : chunk_squares<kF16>(t.in[k], t.n[k], base);
    }
    s = group_total64(s, slot);
    if (threadIdx.x == 0) partial[blockIdx.x] = add ? partial[blockIdx.x] + s : s;
}

template <int DT>
__device__ __forceinline__ void scale_chunk(const Table& t, int k, size_t base, float f)
{
    constexpr int E = Elem<DT>::per16;
    const size_t n = t.n[k];
    u32x4 u[4];
    load_chunk<DT>(t.in[k], base, n, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t at = base + (size_t)(i * kThreads + threadIdx.x) * E;
        float v[E];
        widen16<DT>(u[i], v);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= f;
        if (t.out_t[k] == DT) {
            store16<DT>(t.out[k], at, n, narrow16<DT>(v));
        } else {
            for (int e = 0; e < E; ++e) {
                if (at + e >= n) break;
                if (t.out_t[k] == kF32) store1<kF32>(t.out[k], at + e, v[e]);
                else if (t.out_t[k] == kBF16) store1<kBF16>(t.out[k], at + e, v[e]);
                else store1<kF16>(t.out[k], at + e, v[e]);
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const Table t, const double* partial, int parts,
                                                              float scale, float max_norm, float eps, float* norm)
{
    __shared__ double slot[kThreads / 64];
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
    const float nrm = (float)(sqrt(group_total64(s, slot)) * (double)fabsf(scale));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = nrm;
    float f = max_norm / (nrm + eps);
    f = (f > 1.0f ? 1.0f : f) * scale;           // a NaN norm stays NaN
    const uint64_t total = t.first[t.count];
    int k = t.count - 1;
    for (uint64_t c = blockIdx.x; c < total; c += gridDim.x) {
        const uint64_t r = total - 1 - c;
        while (r < t.first[k]) --k;
        if (f == 1.0f && t.in[k] == t.out[k]) continue;   // in place, times one
        const size_t base = (r - t.first[k]) * chunk_elems(t.in_t[k]);
        if (t.in_t[k] == kF32) scale_chunk<kF32>(t, k, base, f);
        else if (t.in_t[k] == kBF16) scale_chunk<kBF16>(t, k, base, f);
        else scale_chunk<kF16>(t, k, base, f);
    }
}

}  // namespace

hipError_t launch_grad_norm_clip(const GradTensor* g, size_t count, float scale, float max_norm, float eps, void* ws,
                                 float* norm, hipStream_t st)
{
    // the launches: every kTable tensors that hold something
    auto table = [&](size_t& at) {
        Table t = {};
        while (at < count && t.count < kTable) {
            const GradTensor& x = g[at++];
            if (x.n == 0) continue;
            const int i = t.count++;
            t.in[i] = x.in; t.out[i] = x.out; t.n[i] = x.n;
            t.in_t[i] = (uint8_t)x.in_t; t.out_t[i] = (uint8_t)x.out_t;
            const uint64_t per = kChunkBytes / (x.in_t == kF32 ? 4 : 2);
            t.first[i + 1] = t.first[i] + (x.n + per - 1) / per;
        }
        return t;
    };
    uint64_t most = 1;
    for (size_t at = 0; at < count;) {
        const Table t = table(at);
        if (t.first[t.count] > most) most = t.first[t.count];
    }
    const unsigned groups = (unsigned)(most < kClipGroups ? most : kClipGroups);
    double* partial = static_cast<double*>(ws);
    size_t at = 0;
    bool first = true;
    do {
        const Table t = table(at);
        hipLaunchKernelGGL(grad_squares_kernel, dim3(groups), dim3(kThreads), 0, st, t, partial, first ? 0 : 1);
        first = false;
    } while (at < count);
    at = 0;
    first = true;
    do {
        const Table t = table(at);
        hipLaunchKernelGGL(grad_scale_kernel, dim3(groups), dim3(kThreads), 0, st, t, partial, (int)groups, scale,
                           max_norm, eps, first ? norm : nullptr);
        first = false;
    } while (at < count);
    return hipGetLastError();
}

}  // namespace rc
