// The norms around a block, with its gate and the scaled residual.
//
// Forward, for every row of d elements (post norm and gate optional):
//   u = w1 y rstd_y,  rstd_y = 1 / sqrt(mean(y^2) + eps)    (u = y without w1)
//   h = alpha r + g u
//   z = w2 h rstd_h,  rstd_h = 1 / sqrt(mean(h^2) + eps)
// z is formed from h before it is rounded.  Backward, from dz and dh (the
// gradient that reaches h beside z), with yn = y rstd_y, hn = h rstd_h:
//   e  = dh + rstd_h (w2 dz - hn mean(w2 dz hn))            (all of h's gradient)
//   dr = alpha e,  b = e g w1,  dy = rstd_y (b - yn mean(b yn))
//   dw2 = sum over rows of dz hn,  dw1 = sum of e g yn,  dg = e w1 yn
//   (summed over rows for a gate of one value per channel)
// All of it in binary32, every output rounded once.  The work is memory-bound:
// 4 (forward) or 6 (backward) elements per value of a row, so each element is
// read once into registers, a workgroup holds a whole row, and only the two
// row sums go through LDS.  1024 lanes have 128 registers each, which rows wider
// than 16384 forward, and than 8192 backward, overrun: the compiler keeps the
// rest in scratch memory (160 to 430 bytes a lane forward; backward 220 to 490
// up to a width of 16384, 970 to 1490 beyond), which costs time.
//
// bf16, forward: 16384 x 8192 197 us (1.07 GB, 5.4 TB/s), 16384 x 4096 100, one
// row of 4096 3.6; with the next row's loads ahead 211 and 104, with 32 elements
// per lane 208 and 117, with 4096 lanes per unit 200 and 105.  Backward: 8192 x
// 4096 91 us (403 MB and 34 of column sums), 8192 x 8192 161, 16384 x 1024 52;
// fp32 with a full gate 2500 x 1999 49, 2500 x 2000 38.  Wide rows: forward 8192 x
// 16384 202, 2048 x 32768 150 (537 MB); backward 4096 x 8192 92, 4096 x 16384 392
// (805 MB both this and the next), 2048 x 32768 1090.
#include "rc_op.hpp"
#include "rc_op_launch.hpp"

namespace rc {
namespace {

// E neighbouring weights from element i (a multiple of E) on, of type WT.
template <int WT, int E>
__device__ __forceinline__ void weights_at(const void* w, uint32_t i, uint32_t d, float* v)
{
    const uint8_t* p = static_cast<const uint8_t*>(w) + (size_t)i * Elem<WT>::size;
    if (i + E <= d) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            if constexpr (WT == kF32) {
                const u32x4 u = reinterpret_cast<const u32x4*>(p)[e / 4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[e + k] = __uint_as_float(u[k]);
            } else {
                const uint2 u = reinterpret_cast<const uint2*>(p)[e / 4];
                v[e] = WT == kBF16 ? bf16lo(u.x) : f16lo(u.x);
                v[e + 1] = WT == kBF16 ? bf16hi(u.x) : f16hi(u.x);
                v[e + 2] = WT == kBF16 ? bf16lo(u.y) : f16lo(u.y);
                v[e + 3] = WT == kBF16 ? bf16hi(u.y) : f16hi(u.y);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = i + e < d ? load1<WT>(w, i + e) : 0.0f;
    }
}

// The weights of a lane's N vectors of E elements, T lanes apart; without
// weights, `otherwise`.
template <int E, int N, int T>
__device__ __forceinline__ void load_weights(const void* w, int dt, uint32_t d, float (&v)[N * E], float otherwise)
{
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const uint32_t i = (j * T + threadIdx.x) * E;
        if (!w) {
#pragma unroll
            for (int e = 0; e < E; ++e) v[j * E + e] = otherwise;
        } else if (dt == kF32) {
            weights_at<kF32, E>(w, i, d, v + j * E);
        } else if (dt == kBF16) {
            weights_at<kBF16, E>(w, i, d, v + j * E);
        } else {
            weights_at<kF16, E>(w, i, d, v + j * E);
        }
    }
}

template <int DT, int T, int N>
__global__ __launch_bounds__(T) void block_norm_kernel(const BlockNorm a)
{
    constexpr int E = Elem<DT>::per16, W = T / 64, EN = E * N;
    __shared__ float slot[2][2][W];
    const uint32_t d = a.d, i0 = threadIdx.x * E;
    const float inv_d = 1.0f / (float)d;
    const bool post = a.post_w != nullptr, full = a.gate_mode == kGateFull;
    float w1[EN], w2[EN];                        // post weight times a channel gate; pre weight
    load_weights<E, N, T>(a.post_w, a.w_t, d, w1, 1.0f);
    load_weights<E, N, T>(a.pre_w, a.w_t, d, w2, 1.0f);
    if (a.gate_mode == kGateChannel) {
        float g[EN];
        load_weights<E, N, T>(a.gate, a.w_t, d, g, 1.0f);
#pragma unroll
        for (int e = 0; e < EN; ++e) w1[e] *= g[e];
    }
    int turn = 0;
    for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const size_t at = row * d * Elem<DT>::size;
        u32x4 uy[N], ur[N], ug[N];
        load_row<DT>(static_cast<const uint8_t*>(a.y) + at, i0, T * E, d, uy);
        load_row<DT>(static_cast<const uint8_t*>(a.r) + at, i0, T * E, d, ur);
        if (full) load_row<DT>(static_cast<const uint8_t*>(a.gate) + at, i0, T * E, d, ug);
        float rstd_y = 1.0f;
        if (post) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float v[E];
                widen16<DT>(uy[j], v);
#pragma unroll
                for (int e = 0; e < E; ++e) s = fmaf(v[e], v[e], s);
            }
            rstd_y = 1.0f / sqrtf(fmaf(group_total<W>(s, slot[turn][0]), inv_d, a.eps));
        }
        float h[EN], s = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float v[E], q[E], g[E];
            widen16<DT>(uy[j], v);
            widen16<DT>(ur[j], q);
            if (full) widen16<DT>(ug[j], g);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float u = v[e] * rstd_y * w1[j * E + e];
                if (full) u *= g[e];
                const float x = fmaf(a.alpha, q[e], u);
                h[j * E + e] = x;
                s = fmaf(x, x, s);
            }
        }
        const float rstd_h = 1.0f / sqrtf(fmaf(group_total<W>(s, slot[turn][1]), inv_d, a.eps));
        uint8_t* ho = static_cast<uint8_t*>(a.h) + at;
        uint8_t* zo = static_cast<uint8_t*>(a.z) + at;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float v[E], q[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[e] = h[j * E + e];
                q[e] = v[e] * rstd_h * w2[j * E + e];
            }
            const size_t i = i0 + (size_t)j * T * E;
            if (i < d) {
                store16<DT>(ho, i, d, narrow16<DT>(v));
                store16<DT>(zo, i, d, narrow16<DT>(q));
            }
        }
        if (a.stats && threadIdx.x == 0) {
            a.stats[row] = rstd_y;
            a.stats[a.rows + row] = rstd_h;
        }
    }
}

// Backward: the column sums stay in registers over a workgroup's rows and go
// to one row of the workspace per workgroup, [2][d]: dz hn, and e yn (times a
// full gate).  A channel gate and the post weight are the same for all rows,
// so dw1 = g * sum(e yn) and dg = w1 * sum(e yn) come from one sum.
template <int DT, int T, int N, bool FULL>
__global__ __launch_bounds__(T) void block_norm_backward_kernel(const BlockNormBackward a)
{
    constexpr int E = Elem<DT>::per16, W = T / 64, EN = E * N;
    __shared__ float slot[2][2][W];
    const uint32_t d = a.d, i0 = threadIdx.x * E;
    const float inv_d = 1.0f / (float)d;
    constexpr bool full = FULL;
    const bool post = a.post_w != nullptr;
    float w1[EN], w2[EN], sum_pre[EN], sum_y[EN];
    load_weights<E, N, T>(a.post_w, a.w_t, d, w1, 1.0f);
    load_weights<E, N, T>(a.pre_w, a.w_t, d, w2, 1.0f);
    if (a.gate_mode == kGateChannel) {
        float g[EN];
        load_weights<E, N, T>(a.gate, a.w_t, d, g, 1.0f);
#pragma unroll
        for (int e = 0; e < EN; ++e) w1[e] *= g[e];
    }
#pragma unroll
    for (int e = 0; e < EN; ++e) sum_pre[e] = sum_y[e] = 0.0f;
    int turn = 0;
    u32x4 uy[N], uh[N], uz[N], ud[N], ug[N], pz[N], ph[N];
    float rstd_y, rstd_h;
    auto ask = [&](size_t row) {                 // the two that a row's first sum needs
        const size_t at = row * d * Elem<DT>::size;
        load_row<DT>(static_cast<const uint8_t*>(a.dz) + at, i0, T * E, d, pz);
        load_row<DT>(static_cast<const uint8_t*>(a.h) + at, i0, T * E, d, ph);
    };
    // wide rows leave room for two workgroups per compute unit, too few to hide all loads: their next row's
    // are in flight during this one (8192 x 4096 93 -> 90 us; narrow rows lose by it: 16384 x 1024 54 -> 55-61)
    constexpr bool AHEAD = T >= 512;
    if (AHEAD) ask(blockIdx.x);
    for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const size_t at = row * d * Elem<DT>::size;
        if (!AHEAD) ask(row);
#pragma unroll
        for (int j = 0; j < N; ++j) { uz[j] = pz[j]; uh[j] = ph[j]; }
        if (a.dh) load_row<DT>(static_cast<const uint8_t*>(a.dh) + at, i0, T * E, d, ud);
        load_row<DT>(static_cast<const uint8_t*>(a.y) + at, i0, T * E, d, uy);
        if (full) load_row<DT>(static_cast<const uint8_t*>(a.gate) + at, i0, T * E, d, ug);
        rstd_y = post ? a.stats[row] : 1.0f; rstd_h = a.stats[a.rows + row];
        if (AHEAD && row + gridDim.x < a.rows) ask(row + gridDim.x);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float z[E], h[E];
            widen16<DT>(uz[j], z);
            widen16<DT>(uh[j], h);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float t = z[e] * (h[e] * rstd_h);
                sum_pre[j * E + e] += t;
                s = fmaf(t, w2[j * E + e], s);
            }
        }
        const float mz = group_total<W>(s, slot[turn][0]) * inv_d;
        float g[EN];                             // e, all of h's gradient
        s = 0.0f;
        uint8_t* dro = static_cast<uint8_t*>(a.dr) + at;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float z[E], h[E], dh[E], y[E], k[E], o[E];
            widen16<DT>(uz[j], z);
            widen16<DT>(uh[j], h);
            widen16<DT>(uy[j], y);
            if (a.dh) widen16<DT>(ud[j], dh);
            if (full) widen16<DT>(ug[j], k);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = rstd_h * fmaf(-(h[e] * rstd_h), mz, z[e] * w2[j * E + e]) + (a.dh ? dh[e] : 0.0f);
                g[j * E + e] = x;
                o[e] = a.alpha * x;
                const float yn = y[e] * rstd_y;
                const float t = x * yn * (full ? k[e] : 1.0f);
                sum_y[j * E + e] += t;
                s = fmaf(t, w1[j * E + e], s);
                k[e] = x * yn * w1[j * E + e];   // a full gate's gradient
            }
            const size_t i = i0 + (size_t)j * T * E;
            if (i < d) {
                store16<DT>(dro, i, d, narrow16<DT>(o));
                if (full && a.dgate) store16<DT>(static_cast<uint8_t*>(a.dgate) + at, i, d, narrow16<DT>(k));
            }
        }
        const float my = post ? group_total<W>(s, slot[turn][1]) * inv_d : 0.0f;
        uint8_t* dyo = static_cast<uint8_t*>(a.dy) + at;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float y[E], k[E], o[E];
            widen16<DT>(uy[j], y);
            if (full) widen16<DT>(ug[j], k);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float b = g[j * E + e] * w1[j * E + e] * (full ? k[e] : 1.0f);
                o[e] = rstd_y * fmaf(-(y[e] * rstd_y), my, b);
            }
            const size_t i = i0 + (size_t)j * T * E;
            if (i < d) store16<DT>(dyo, i, d, narrow16<DT>(o));
        }
    }
    float* part = a.partial + (size_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int e = 0; e < EN; ++e) {
        const uint32_t i = (e / E * T + threadIdx.x) * E + e % E;
        if (i < d) { part[i] = sum_pre[e]; part[d + i] = sum_y[e]; }
    }
}

// Adds the workgroups' column sums: 64 of the workspace's 2 d columns per
// workgroup, its 16 waves each a run of its rows (eight loads in flight), then
// the waves' sums in order.  Columns d .. 2 d - 1 give dw1 and a channel
// gate's gradient.
__global__ __launch_bounds__(1024) void block_norm_columns_kernel(const BlockNormBackward a, int parts)
{
    __shared__ float sums[16][64];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d = a.d, width = 2 * d;
    const uint32_t c = blockIdx.x * 64 + lane, run = (parts + 15) / 16, first = wave * run, last = min(first + run, (uint32_t)parts);
    float s = 0.0f;
    if (c < width) {
        const float* p = a.partial + (size_t)first * width + c;
        uint32_t k = first;
        for (; k + 8 <= last; k += 8, p += (size_t)8 * width) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[(size_t)i * width];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; k < last; ++k, p += width) s += *p;
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= width) return;
    s = sums[0][lane];
#pragma unroll
    for (int w = 1; w < 16; ++w) s += sums[w][lane];
    if (c < d) {
        a.dpre[c] = s;
        return;
    }
    const uint32_t i = c - d;
    const bool channel = a.gate_mode == kGateChannel;
    if (a.dpost) a.dpost[i] = channel ? s * load1_rt(a.gate, a.w_t, i) : s;
    if (channel && a.dgate) static_cast<float*>(a.dgate)[i] = a.post_w ? s * load1_rt(a.post_w, a.w_t, i) : s;
}

// f(threads, vectors per lane) for rows of d elements, EPT elements per lane
// while 1024 lanes suffice.  Forward 8 up to a width of 4096 and 16 beyond
// (16384 x 4096 100 us and 107, 16384 x 8192 214 and 197); backward 8, for the
// registers of the column sums.
template <int DT, int EPT, class F>
hipError_t with_shape(uint32_t d, F&& f)
{
    constexpr int E = Elem<DT>::per16, N = EPT / E;
    using std::integral_constant;
#define RC_SHAPE(T, V) return f(integral_constant<int, T>{}, integral_constant<int, V>{})
    if (d <= 64 * EPT) RC_SHAPE(64, N);
    if (d <= 128 * EPT) RC_SHAPE(128, N);
    if (d <= 256 * EPT) RC_SHAPE(256, N);
    if (d <= 512 * EPT) RC_SHAPE(512, N);
    if (d <= 1024 * EPT) RC_SHAPE(1024, N);
    if constexpr (EPT < 16) if (d <= 1024 * 16) RC_SHAPE(1024, 16 / E);
    RC_SHAPE(1024, 32 / E);
#undef RC_SHAPE
}

template <int DT>
hipError_t forward_t(const BlockNorm& a, hipStream_t st)
{
    const auto launch = [&](auto t, auto n) {
        const size_t most = (size_t)compute_units() * ((t >= 512 ? 1024 : 2048) / t);
        hipLaunchKernelGGL((block_norm_kernel<DT, t, n>), dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(t), 0, st, a);
        return hipGetLastError();
    };
    return a.d <= 4096 ? with_shape<DT, 8>(a.d, launch) : with_shape<DT, 16>(a.d, launch);
}

template <int DT>
hipError_t backward_t(const BlockNormBackward& a, unsigned groups, hipStream_t st)
{
    const auto launch = [&](auto t, auto n) {
        if (groups && a.gate_mode == kGateFull) hipLaunchKernelGGL((block_norm_backward_kernel<DT, t, n, true>), dim3(groups), dim3(t), 0, st, a);
        else if (groups) hipLaunchKernelGGL((block_norm_backward_kernel<DT, t, n, false>), dim3(groups), dim3(t), 0, st, a);
        hipLaunchKernelGGL(block_norm_columns_kernel, dim3((2 * a.d + 63) / 64), dim3(1024), 0, st, a, (int)groups);
        return hipGetLastError();
    };
    return with_shape<DT, 8>(a.d, launch);
}

}  // namespace

hipError_t launch_block_norm(int dt, const BlockNorm& a, hipStream_t st)
{
    return dt == kF32 ? forward_t<kF32>(a, st) : dt == kF16 ? forward_t<kF16>(a, st) : forward_t<kBF16>(a, st);
}

hipError_t launch_block_norm_backward(int dt, const BlockNormBackward& a, hipStream_t st)
{
    const unsigned groups = block_norm_groups(a.rows, a.d);
    return dt == kF32 ? backward_t<kF32>(a, groups, st)
         : dt == kF16 ? backward_t<kF16>(a, groups, st) : backward_t<kBF16>(a, groups, st);
}

}  // namespace rc
