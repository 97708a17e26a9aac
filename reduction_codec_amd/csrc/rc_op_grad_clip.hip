// Global norm of many tensors, and clipping by it.
//
//   N = |scale| sqrt(sum over all tensors of g^2)
//   out = round(g * scale * min(1, max_norm / (N + eps)))   (max_norm infinite: g * scale)
//
// Two kernels read the tensors through a table in the kernel arguments (no
// device copy of the pointers, so a call can be captured and replayed).  Every
// tensor is cut into 16 KiB chunks; a workgroup takes the chunks of all the
// table's tensors with a stride of the grid, finds each by bisection, and keeps
// one sum of squares, in binary64: the squares of binary32 values neither
// overflow nor vanish there, and the order of the additions, fixed by the
// sizes and the first kernel's alignment alone, does not show in the rounded
// norm.  The second kernel adds the workgroups' sums (each of its workgroups
// for itself, 8 KiB from L2, which saves a launch and a wait) and scales the
// chunks from the last to the first, so that what the first kernel read last
// is still in the 256 MiB cache; its stores do not go there.
//
// Bound by memory: two reads and a write.  805 M bf16 values into others 876 -
// 892 us (4.8 GB, 5.4 - 5.5 TB/s), in place 744, 30 M fp16 values in 104 tensors at odd places 40 us, 1.8 M
// fp32 in 48 tensors 10.5 us, of which half are the two launches.  Measured
// against: 2048 workgroups 901 us, 8 or 2 loads per lane 909, 923, cached
// stores 902, uncached loads in the second pass 852 but 42 and 11.4 us for the
// smaller ones; a walk through the table instead of the bisection 60 and 14.6.
#include "rc_op.hpp"
#include "rc_op_launch.hpp"

namespace rc {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                         // 16-byte loads per lane and chunk
constexpr uint32_t kChunkBytes = kThreads * kVecs * 16;
constexpr int kTable = 116;                      // tensors per launch: 31 bytes of kernel arguments each, under 4 KiB in all

struct Table {
    const uint8_t* in[kTable];                   // both `lead` elements before the tensor's first
    uint8_t* out[kTable];
    uint64_t n[kTable];
    uint32_t first[kTable + 1];                  // first chunk of each tensor, total last
    uint8_t in_t[kTable], out_t[kTable], lead[kTable];
    int count;
};

// The tensor of chunk c, starting from a guess.
__device__ __forceinline__ int tensor_of(const Table& t, uint32_t c, int k)
{
    if (c >= t.first[k] && c < t.first[k + 1]) return k;
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (c >= t.first[mid]) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

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

// A chunk's elements are counted from the 16-byte boundary at or before the
// tensor's first one (`lead` elements before it), so whole chunks are read
// aligned wherever the tensor starts; [lead, end) holds the tensor.
template <int DT>
__device__ __forceinline__ void load_chunk(const uint8_t* in, size_t base, uint32_t lead, size_t end, u32x4 (&u)[kVecs])
{
    constexpr int E = Elem<DT>::per16, S = Elem<DT>::size;
    const size_t i = base + threadIdx.x * E;
    if (base >= lead && base + chunk_elems(DT) <= end) {         // uniform: all but the first and the last
#pragma unroll
        for (int j = 0; j < kVecs; ++j) u[j] = *reinterpret_cast<const u32x4*>(in + (i + j * kThreads * E) * S);
    } else {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const size_t k = i + j * kThreads * E;
            u[j] = u32x4{0, 0, 0, 0};
            if (k >= lead && k + E <= end) {
                u[j] = *reinterpret_cast<const u32x4*>(in + k * S);
            } else if (k + E > lead && k < end) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (k + e < lead || k + e >= end) continue;
                    if constexpr (S == 4) u[j][e] = reinterpret_cast<const uint32_t*>(in)[k + e];
                    else u[j][e / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(in)[k + e] << (16 * (e % 2));
                }
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ double chunk_squares(const Table& t, int k, size_t base)
{
    constexpr int E = Elem<DT>::per16;
    u32x4 u[kVecs];
    load_chunk<DT>(t.in[k], base, t.lead[k], t.lead[k] + t.n[k], u);
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
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
    for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        k = tensor_of(t, c, k);
        const size_t base = (size_t)(c - t.first[k]) * chunk_elems(t.in_t[k]);
        s += t.in_t[k] == kF32 ? chunk_squares<kF32>(t, k, base)
           : t.in_t[k] == kBF16 ? chunk_squares<kBF16>(t, k, base)
                                : chunk_squares<kF16>(t, k, base);
    }
    s = group_total64(s, slot);
    if (threadIdx.x == 0) partial[blockIdx.x] = add ? partial[blockIdx.x] + s : s;
}

template <int DT, int OT>
__device__ __forceinline__ void store_scaled(uint8_t* out, size_t k, uint32_t lead, size_t end, u32x4 u, float f)
{
    constexpr int E = Elem<DT>::per16;
    float v[E];
    widen16<DT>(u, v);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= f;
    if (OT == DT && k >= lead && k + E <= end) {
        __builtin_nontemporal_store(narrow16<DT>(v), reinterpret_cast<u32x4_any*>(out + k * Elem<DT>::size));
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (k + e >= lead && k + e < end) store1<OT>(out, k + e, v[e]);
    }
}

template <int DT>
__device__ __forceinline__ void scale_chunk(const Table& t, int k, size_t base, float f)
{
    constexpr int E = Elem<DT>::per16;
    const uint32_t lead = t.lead[k];
    const size_t end = lead + t.n[k];
    u32x4 u[kVecs];
    load_chunk<DT>(t.in[k], base, lead, end, u);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const size_t at = base + (size_t)(i * kThreads + threadIdx.x) * E;
        if (t.out_t[k] == kF32) store_scaled<DT, kF32>(t.out[k], at, lead, end, u[i], f);
        else if (t.out_t[k] == kBF16) store_scaled<DT, kBF16>(t.out[k], at, lead, end, u[i], f);
        else store_scaled<DT, kF16>(t.out[k], at, lead, end, u[i], f);
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
    f = (f > 1.0f || isinf(max_norm) ? 1.0f : f) * scale;   // a NaN norm stays NaN, but no limit clips nothing
    const uint32_t total = t.first[t.count];
    int k = 0;
    for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
        const uint32_t r = total - 1 - c;
        k = tensor_of(t, r, k);
        // in place, times one: one type too, for both addresses lie `lead` elements of their own types back
        if (f == 1.0f && t.in[k] == t.out[k] && t.in_t[k] == t.out_t[k]) continue;
        const size_t base = (size_t)(r - t.first[k]) * chunk_elems(t.in_t[k]);
        if (t.in_t[k] == kF32) scale_chunk<kF32>(t, k, base, f);
        else if (t.in_t[k] == kBF16) scale_chunk<kBF16>(t, k, base, f);
        else scale_chunk<kF16>(t, k, base, f);
    }
}

}  // namespace

hipError_t launch_grad_norm_clip(const GradTensor* g, size_t count, float scale, float max_norm, float eps, void* ws,
                                 float* norm, hipStream_t st)
{
    // the launches: every kTable tensors that hold something (2^40 elements are 2^28 chunks at most)
    auto table = [&](size_t& at) {
        Table t = {};
        while (at < count && t.count < kTable) {
            const GradTensor& x = g[at++];
            if (x.n == 0) continue;
            if (t.first[t.count] >= 1u << 30) { --at; break; }
            const int i = t.count++;
            const uint32_t size = x.in_t == kF32 ? 4 : 2, lead = (uint32_t)(reinterpret_cast<uintptr_t>(x.in) % 16) / size;
            t.in[i] = static_cast<const uint8_t*>(x.in) - lead * size;
            t.out[i] = static_cast<uint8_t*>(x.out) - lead * (x.out_t == kF32 ? 4 : 2);
            t.n[i] = x.n;
            t.in_t[i] = (uint8_t)x.in_t; t.out_t[i] = (uint8_t)x.out_t; t.lead[i] = (uint8_t)lead;
            const uint64_t per = kChunkBytes / size;
            t.first[i + 1] = t.first[i] + (uint32_t)((lead + x.n + per - 1) / per);
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
