// New tokens into a paged cache held in MXFP4, turned by their positions on the
// way, and the rows read back.
//
// A lane has eight values of a row, a quad of lanes a block of 32: its maximum
// is two lane swaps away, its codes are four neighbouring words.  A turned
// value a cos - b sin is formed in binary64, where it is right to the last bit
// (both products of a 24-bit value and a 24-bit angle are exact), so that the
// codes are those of the value itself: the scale is the exponent of the block's
// maximum, and what 21 bits of x drop is kept as their last bit, from where the
// rounding to four bits goes the way that the value itself would.
#include "rc_op_cache.hpp"
#include "rc_op_rules.hpp"

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

// ONCE: nobody reads them again (past the caches, 12288 tokens are appended in 55
// us, 59 through them).
template <int DT, bool ONCE = false>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8])
{
    const u32x4* const at = reinterpret_cast<const u32x4*>(p);
    const auto load = [&](int i) { return ONCE ? __builtin_nontemporal_load(at + i) : at[i]; };
    if constexpr (DT == kF32) {
        const u32x4 a = load(0), b = load(1);
        for (int e = 0; e < 4; ++e) { v[e] = __uint_as_float(a[e]); v[4 + e] = __uint_as_float(b[e]); }
    } else {
        widen8<DT>(load(0), v);
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

// Lanes of a workgroup where units go one by one; kTokenLanes where it takes a token.
constexpr int kAppendLanes = 256;

// The upper half of |y| with its last bit set where the lower half holds
// anything: 21 bits, from where any rounding to 19 or fewer is right.
__device__ __forceinline__ uint32_t odd_half(double y)
{
    const uint64_t u = (uint64_t)__double_as_longlong(y);
    const uint32_t lo = (uint32_t)u;
    return ((uint32_t)(u >> 32) & 0x7FFFFFFF) | (lo < 1 ? lo : 1);
}

// The codes of eight values of a block whose largest is 2^(ex + 2) and more:
// y 2^-ex in binary32, its exponent moved among integers (what falls below
// 2^-126 is 0 as a code, what passes the range is the largest).
__device__ __forceinline__ uint32_t codes8(const double (&y)[8], int ex)
{
    const uint32_t shift = (uint32_t)(1023 - 127 + ex) << 20;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t m = odd_half(y[e]), n = __builtin_elementwise_sub_sat(m, shift), top = n < 0x0FEFFFFF ? n : 0x0FEFFFFF;
        f[e] = __uint_as_float((top << 3 & 0x7FFFFFFF) | ((uint32_t)(__double_as_longlong(y[e]) >> 32) & 0x80000000));
    }
    uint32_t w = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) w = fp4_enc(w, f[2 * b], f[2 * b + 1], 1.0f, b);
    return w;
}

// Eight values for one rounding to DT.  Those of 21 bits are exact in binary32
// but below its range, where binary32 rounds and the odd bit is set from there.
template <int DT>
__device__ __forceinline__ void round8(const double (&y)[8], float (&v)[8])
{
    if constexpr (DT == kF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)y[e];
        return;
    }
    float least = INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint64_t u = (uint64_t)__double_as_longlong(y[e]);
        const uint32_t lo = (uint32_t)u;
        v[e] = (float)__longlong_as_double((long long)((uint64_t)((uint32_t)(u >> 32) | (lo < 1 ? lo : 1)) << 32));
        least = __builtin_fminf(least, __builtin_fabsf(v[e]));
    }
    if (__builtin_amdgcn_ballot_w64(least < 0x1p-126f) == 0) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = round_odd(y[e]);
}

// Upper halves of binary64 order magnitudes as their exponents do.
__device__ __forceinline__ uint32_t largest8(const double (&y)[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t m = (uint32_t)(__double_as_longlong(y[e]) >> 32) & 0x7FFFFFFF;
        top = top > m ? top : m;
    }
    return top;
}

__device__ __forceinline__ int exponent_of(uint32_t top)
{
    const int ex = (int)(top >> 20) - 1023 - 2;
    return ex < -127 ? -127 : ex > 127 ? 127 : ex;
}

// The token of a workgroup, and a grid of `y` workgroups for each: a grid's x is
// at most 2^32 lanes, so z takes what is more.
constexpr unsigned kTokensOfX = 1u << 22;
__device__ __forceinline__ unsigned token_of_block() { return blockIdx.z * gridDim.x + blockIdx.x; }
dim3 grid_of_tokens(int tokens, unsigned y)
{
    const unsigned n = (unsigned)tokens, x = n < kTokensOfX ? n : kTokensOfX;
    return dim3(x, y, (n + x - 1) / x);
}

// A lane has two units of eight values of a head that are turned together, and
// those of every (kTokenLanes / (D / 16))-th head, so that a token's angles are
// read once: units u and u + rot / 16 of the first rot values (or neighbours if
// interleaved), neighbours of the rest, and of values.  A block is four units: of
// neighbouring lanes' first units, or second ones, or both of two lanes.  That
// takes rot to be a multiple of 64 (or neighbours) and D of 64; what is not goes
// unit by unit below.  12288 tokens of 48 heads of 128, bf16 (265 MB): 55 us, 4.8
// TB/s; 89 us unit by unit, where every head reads the angles and half of it
// twice.  The loads of a token wait for its place and one another, so that the
// kernel is bound by how many tokens are in flight: values asked for ahead cost
// registers and with them waves (64 to 67 us, against 59), and neighbouring tokens on one XCD,
// whose codes share lines, change nothing.
template <int DT, int D>
__global__ __launch_bounds__(kTokenLanes) void cache_append_pairs_kernel(const CacheAppend a)
{
    constexpr int I = D / 16, ES = Elem<DT>::size, HP = kTokenLanes / I;
    const int token = (int)token_of_block(), kv = a.c.kv_heads, all = a.heads + 2 * kv, item = threadIdx.x % I;
    if ((unsigned)token >= (unsigned)a.c.tokens) return;
    const RowPlace at = row_place(a.c, token);
    if (at.seq < 0 || threadIdx.x >= HP * I) return;
    const int page = page_of(a.c, at.seq, at.pos), half = a.rot / 2;
    const bool turned = item * 16 < a.rot, split = turned && !a.interleaved;
    double cs[8], sn[8];
    if (turned) {
        const float* turn = a.rotation + (size_t)(at.pos < 0 ? 0 : at.pos) * a.rot + item * 8;
        float c[8], s[8];
        load8<kF32>(reinterpret_cast<const uint8_t*>(turn), c);
        load8<kF32>(reinterpret_cast<const uint8_t*>(turn + half), s);
#pragma unroll
        for (int e = 0; e < 8; ++e) { cs[e] = c[e]; sn[e] = s[e]; }
    }
    for (int row = blockIdx.y * HP + threadIdx.x / I; row < all; row += gridDim.y * HP) {
        const bool query = row < a.heads, value = row >= a.heads + kv, both = split && !value;
        const int head = row - (query ? 0 : value ? a.heads + kv : a.heads);
        const uint8_t* src = static_cast<const uint8_t*>(query ? a.q : value ? a.v : a.k) +
                             ((size_t)token * (query ? a.q_stride : value ? a.v_stride : a.k_stride) + (size_t)head * D) * ES;
        // the units of this lane
        const int u0 = both ? item : 2 * item, u1 = both ? item + half / 8 : 2 * item + 1;
        float v0[8], v1[8];
        load8<DT, true>(src + u0 * 8 * ES, v0);
        load8<DT, true>(src + u1 * 8 * ES, v1);
        double y0[8], y1[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) { y0[e] = v0[e]; y1[e] = v1[e]; }
        if (both) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double p = y0[e], q = y1[e];
                y0[e] = __builtin_fma(q, -sn[e], p * cs[e]);
                y1[e] = __builtin_fma(p, sn[e], q * cs[e]);
            }
        } else if (turned && !value) {           // neighbours
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const double p = y0[2 * e], q = y0[2 * e + 1], r = y1[2 * e], s = y1[2 * e + 1];
                y0[2 * e] = __builtin_fma(q, -sn[e], p * cs[e]);
                y0[2 * e + 1] = __builtin_fma(p, sn[e], q * cs[e]);
                y1[2 * e] = __builtin_fma(s, -sn[4 + e], r * cs[4 + e]);
                y1[2 * e + 1] = __builtin_fma(r, sn[4 + e], s * cs[4 + e]);
            }
        }
        if (query) {
            round8<DT>(y0, v0);
            round8<DT>(y1, v1);
            uint8_t* out = static_cast<uint8_t*>(a.q_out) + ((size_t)token * a.heads + head) * D * ES;
            store8<DT>(out + u0 * 8 * ES, v0);
            store8<DT>(out + u1 * 8 * ES, v1);
            continue;
        }
        const uint32_t t0 = largest8(y0), t1 = largest8(y1), t = t0 > t1 ? t0 : t1;
        const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0xB1, 0xF, 0xF, false);     // the lane beside
        const int ex0 = exponent_of(both ? quad_max(t0) : t > other ? t : other), ex1 = both ? exponent_of(quad_max(t1)) : ex0;
        const uint32_t w0 = codes8(y0, ex0), w1 = codes8(y1, ex1);
        if (page < 0) continue;
        uint8_t* out = (value ? a.c.v : a.c.k) + stream_at(a.c, page, head);
        const uint32_t block = (uint32_t)(at.pos & ((1 << a.c.shift) - 1)) * (D / 32);
        *reinterpret_cast<uint32_t*>(out + codes_at(block + u0 / 4) + u0 % 4 * 4) = w0;
        *reinterpret_cast<uint32_t*>(out + codes_at(block + u1 / 4) + u1 % 4 * 4) = w1;
        if (u0 % 4 == 0) out[scale_at(block + u0 / 4)] = (uint8_t)(ex0 + 127);
        if (both && u1 % 4 == 0) out[scale_at(block + u1 / 4)] = (uint8_t)(ex1 + 127);
    }
}

// Unit by unit: one token a row of the grid; blockIdx.y cuts its heads (q, k, v).
template <int DT, int D>
__global__ __launch_bounds__(kAppendLanes) void cache_append_kernel(const CacheAppend a)
{
    constexpr int U = D / 8, ES = Elem<DT>::size;
    const int token = (int)token_of_block(), kv = a.c.kv_heads, unit = blockIdx.y * kAppendLanes + threadIdx.x;
    int head = unit / U;
    const int c = unit % U;
    if ((unsigned)token >= (unsigned)a.c.tokens) return;
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
                y[2 * e] = __builtin_fma(q, -sn, p * cs);
                y[2 * e + 1] = __builtin_fma(p, sn, q * cs);
            }
        } else {
            const bool second = c * 8 >= half;
            const int i = second ? c * 8 - half : c * 8;
            float w[8];
            load8<DT>(row + (second ? i : i + half) * ES, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double cs = turn[i + e], sn = second ? turn[half + i + e] : -turn[half + i + e];
                y[e] = __builtin_fma((double)w[e], sn, y[e] * cs);
            }
        }
    }
    if (query) {
        round8<DT>(y, v);
        store8<DT>(static_cast<uint8_t*>(a.q_out) + (((size_t)token * a.heads + head) * D + c * 8) * ES, v);
        return;
    }
    const int ex = exponent_of(quad_max(largest8(y)));
    const uint32_t w = codes8(y, ex);
    const int page = page_of(a.c, at.seq, at.pos);
    if (page < 0) return;
    uint8_t* out = (value ? a.c.v : a.c.k) + stream_at(a.c, page, head);
    const uint32_t block = (uint32_t)(at.pos & ((1 << a.c.shift) - 1)) * (D / 32) + c / 4;
    *reinterpret_cast<uint32_t*>(out + codes_at(block) + c % 4 * 4) = w;
    if (c % 4 == 0) out[scale_at(block)] = (uint8_t)(ex + 127);
}

template <int DT, int D>
__global__ __launch_bounds__(kTokenLanes) void cache_read_kernel(const Cache c, void* k, void* v)
{
    constexpr int U = D / 8, ES = Elem<DT>::size;
    const int token = (int)token_of_block(), units = 2 * U * c.kv_heads;
    if ((unsigned)token >= (unsigned)c.tokens) return;
    const RowPlace at = row_place(c, token);
    if (at.seq < 0) return;
    const int page = page_of(c, at.seq, at.pos);
    for (int unit = blockIdx.y * kTokenLanes + threadIdx.x; unit < units; unit += gridDim.y * kTokenLanes) {
        const int i = unit % U;
        const bool value = unit >= U * c.kv_heads;
        const int head = unit / U - (value ? c.kv_heads : 0);
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
}

template <int DT, int D>
hipError_t append_t(const CacheAppend& a, hipStream_t st)
{
    if constexpr (D % 64 == 0) {
        if (append_in_pairs(D, (unsigned)a.rot, a.interleaved)) {
            const unsigned y = side_by_side(a.c.tokens, append_turns((unsigned)(a.heads + 2 * a.c.kv_heads), D));
            cache_append_pairs_kernel<DT, D><<<grid_of_tokens(a.c.tokens, y), kTokenLanes, 0, st>>>(a);
            return hipGetLastError();
        }
    }
    const unsigned y = ((unsigned)(a.heads + 2 * a.c.kv_heads) * (D / 8) + kAppendLanes - 1) / kAppendLanes;
    cache_append_kernel<DT, D><<<grid_of_tokens(a.c.tokens, y), kAppendLanes, 0, st>>>(a);
    return hipGetLastError();
}

template <int DT, int D>
hipError_t read_t(const Cache& c, void* k, void* v, hipStream_t st)
{
    const unsigned y = side_by_side(c.tokens, read_turns((unsigned)c.kv_heads, D));
    cache_read_kernel<DT, D><<<grid_of_tokens(c.tokens, y), kTokenLanes, 0, st>>>(c, k, v);
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
