// New tokens into a paged cache held in MXFP4, turned by their positions on the
// way, and the rows read back.
//
// A lane has eight values of a row, a quad of lanes a block of 32: its maximum
// is two lane swaps away, its codes are four neighbouring words.  A turned
// value a cos - b sin is formed in binary64, where it is right to the last bit
// (both products of a 24-bit value and a 24-bit angle are exact), so that the
// codes are those of the value itself: the scale is the exponent of the block's
// maximum, and x 2^-e, exact, is rounded to odd in binary32, from where the
// rounding to four bits goes the way that the value itself would.
#include "rc_op_cache.hpp"

namespace rc {
namespace {

// Rounded to binary32 with the last bit set where anything is lost, so that a
// second rounding to fewer than 23 bits is right.
__device__ __forceinline__ float round_odd(double x)
{
    const float f = (float)x;
    const double back = f;
    uint32_t u = __float_as_uint(f);
    if (__builtin_fabs(back) > __builtin_fabs(x)) --u;
    if (back != x) u |= 1;
    return __uint_as_float(u);
}

template <int DT>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8])
{
    if constexpr (DT == kF32) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(p), b = *reinterpret_cast<const u32x4*>(p + 16);
        for (int e = 0; e < 4; ++e) { v[e] = __uint_as_float(a[e]); v[4 + e] = __uint_as_float(b[e]); }
    } else {
        widen8<DT>(*reinterpret_cast<const u32x4*>(p), v);
    }
}

template <int DT>
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[8])
{
    if constexpr (DT == kF32) {
        const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
        *reinterpret_cast<u32x4*>(p) = narrow16<DT>(a);
        *reinterpret_cast<u32x4*>(p + 16) = narrow16<DT>(b);
    } else {
        *reinterpret_cast<u32x4*>(p) = narrow16<DT>(v);
    }
}

// Maximum over a quad of lanes, in each of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false);
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false);
    return v > o ? v : o;
}

constexpr int kAppendLanes = 256;

// One token a workgroup row of the grid; blockIdx.y cuts its heads (q, k, v).
template <int DT, int D>
__global__ __launch_bounds__(kAppendLanes) void cache_append_kernel(const CacheAppend a)
{
    constexpr int U = D / 8, ES = Elem<DT>::size;
    const int token = blockIdx.x, kv = a.c.kv_heads, unit = blockIdx.y * kAppendLanes + threadIdx.x;
    int head = unit / U;
    const int c = unit % U;
    const RowPlace at = row_place(a.c, token);
    if (at.seq < 0 || head >= a.heads + 2 * kv) return;
    const bool query = head < a.heads, value = head >= a.heads + kv;
    const void* src = query ? a.q : value ? a.v : a.k;
    const size_t stride = query ? a.q_stride : value ? a.v_stride : a.k_stride;
    head -= query ? 0 : value ? a.heads + kv : a.heads;
    const uint8_t* row = static_cast<const uint8_t*>(src) + ((size_t)token * stride + (size_t)head * D) * ES;

    float v[8];
    double y[8];
    load8<DT>(row + c * 8 * ES, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = v[e];
    const int half = a.rot / 2;
    if (!value && c * 8 < a.rot) {
        const float* turn = a.rotation + (size_t)(at.pos < 0 ? 0 : at.pos) * a.rot;
        if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const double cs = turn[c * 4 + e], sn = turn[half + c * 4 + e];
                const double p = y[2 * e], q = y[2 * e + 1];
                y[2 * e] = p * cs - q * sn;
                y[2 * e + 1] = q * cs + p * sn;
            }
        } else {
            const bool second = c * 8 >= half;
            const int i = second ? c * 8 - half : c * 8;
            float w[8];
            load8<DT>(row + (second ? i : i + half) * ES, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double cs = turn[i + e], sn = second ? turn[half + i + e] : -turn[half + i + e];
                y[e] = y[e] * cs + (double)w[e] * sn;
            }
        }
    }
    if (query) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = DT == kF32 ? (float)y[e] : round_odd(y[e]);
        store8<DT>(static_cast<uint8_t*>(a.q_out) + (((size_t)token * a.heads + head) * D + c * 8) * ES, v);
        return;
    }
    uint32_t top = 0;                            // upper halves order magnitudes as their exponents do
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t m = (uint32_t)(__double_as_longlong(y[e]) >> 32) & 0x7FFFFFFF;
        top = top > m ? top : m;
    }
    int ex = (int)(quad_max(top) >> 20) - 1023 - 2;
    ex = ex < -127 ? -127 : ex > 127 ? 127 : ex;
    uint32_t w = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
        w = fp4_enc(w, round_odd(__builtin_ldexp(y[2 * b], -ex)), round_odd(__builtin_ldexp(y[2 * b + 1], -ex)), 1.0f, b);
    const int page = page_of(a.c, at.seq, at.pos);
    if (page < 0) return;
    uint8_t* out = (value ? a.c.v : a.c.k) + stream_at(a.c, page, head);
    const uint32_t block = (uint32_t)(at.pos & ((1 << a.c.shift) - 1)) * (D / 32) + c / 4;
    *reinterpret_cast<uint32_t*>(out + codes_at(block) + c % 4 * 4) = w;
    if (c % 4 == 0) out[scale_at(block)] = (uint8_t)(ex + 127);
}

template <int DT, int D>
__global__ __launch_bounds__(kAppendLanes) void cache_read_kernel(const Cache c, void* k, void* v)
{
    constexpr int U = D / 8, ES = Elem<DT>::size;
    const int token = blockIdx.x, unit = blockIdx.y * kAppendLanes + threadIdx.x;
    const int head = unit / U % c.kv_heads, i = unit % U;
    const bool value = unit >= U * c.kv_heads;
    const RowPlace at = row_place(c, token);
    if (at.seq < 0 || unit >= 2 * U * c.kv_heads) return;
    const int page = page_of(c, at.seq, at.pos);
    float x[8] = {};
    if (page >= 0) {
        const uint8_t* in = (value ? c.v : c.k) + stream_at(c, page, head);
        const uint32_t block = (uint32_t)(at.pos & ((1 << c.shift) - 1)) * (D / 32) + i / 4;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(in + codes_at(block) + i % 4 * 4);
        const float s = __uint_as_float((uint32_t)in[scale_at(block)] << 23);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const f2 p = fp4_dec(w, s, b);
            x[2 * b] = p.x;
            x[2 * b + 1] = p.y;
        }
    }
    store8<DT>(static_cast<uint8_t*>(value ? v : k) + (((size_t)token * c.kv_heads + head) * D + i * 8) * ES, x);
}

template <int DT, int D>
hipError_t append_t(const CacheAppend& a, hipStream_t st)
{
    const unsigned y = ((unsigned)(a.heads + 2 * a.c.kv_heads) * (D / 8) + kAppendLanes - 1) / kAppendLanes;
    cache_append_kernel<DT, D><<<dim3((unsigned)a.c.tokens, y), kAppendLanes, 0, st>>>(a);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t read_t(const Cache& c, void* k, void* v, hipStream_t st)
{
    const unsigned y = ((unsigned)c.kv_heads * 2 * (D / 8) + kAppendLanes - 1) / kAppendLanes;
    cache_read_kernel<DT, D><<<dim3((unsigned)c.tokens, y), kAppendLanes, 0, st>>>(c, k, v);
    return hipGetLastError();
}

template <int DT>
hipError_t append_d(int d, const CacheAppend& a, hipStream_t st)
{
    switch (d) {
    case 64: return append_t<DT, 64>(a, st);
    case 96: return append_t<DT, 96>(a, st);
    case 128: return append_t<DT, 128>(a, st);
    case 192: return append_t<DT, 192>(a, st);
    default: return append_t<DT, 256>(a, st);
    }
}

template <int DT>
hipError_t read_d(int d, const Cache& c, void* k, void* v, hipStream_t st)
{
    switch (d) {
    case 64: return read_t<DT, 64>(c, k, v, st);
    case 96: return read_t<DT, 96>(c, k, v, st);
    case 128: return read_t<DT, 128>(c, k, v, st);
    case 192: return read_t<DT, 192>(c, k, v, st);
    default: return read_t<DT, 256>(c, k, v, st);
    }
}

}  // namespace

hipError_t launch_cache_append(int dt, int d, const CacheAppend& a, hipStream_t st)
{
    return dt == kF32 ? append_d<kF32>(d, a, st) : dt == kF16 ? append_d<kF16>(d, a, st) : append_d<kBF16>(d, a, st);
}

hipError_t launch_cache_read(int dt, int d, const Cache& c, void* k, void* v, hipStream_t st)
{
    return dt == kF32 ? read_d<kF32>(d, c, k, v, st) : dt == kF16 ? read_d<kF16>(d, c, k, v, st) : read_d<kBF16>(d, c, k, v, st);
}

}  // namespace rc
