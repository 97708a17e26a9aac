// rc_op.hpp -- device helpers shared by the operators around the codec:
// 16-byte vectors of any element type, widened to binary32 and rounded back
// once, and sums over a wave and over a workgroup.
#pragma once

#include "rc_device.hpp"

namespace rc {

// 16 bytes at any element-aligned address (gfx950 global accesses need no
// 16-byte alignment; rows of odd width and tensors cut from one buffer start
// anywhere).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16_pair __attribute__((ext_vector_type(2)));
typedef _Float16 f16_pair __attribute__((ext_vector_type(2)));

// A buffer descriptor for `bytes` bytes at base + off: offsets past them read
// as zeros and move nothing.
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc span_rsrc(const void* base, size_t off, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void*)(static_cast<const uint8_t*>(base) + off), (short)0, (int)bytes, 0x00020000);
}

template <int DT> struct Elem { static constexpr int size = (DT == kF32) ? 4 : 2, per16 = 16 / size; };

// The elements of 16 bytes, widened exactly.
template <int DT>
__device__ __forceinline__ void widen16(const u32x4 u, float (&v)[Elem<DT>::per16])
{
    if constexpr (DT == kF32) {
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    } else {
        widen8<DT>(u, v);
    }
}

// Two binary32 values rounded to nearest even into one word.
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float a, float b)
{
    const f32x2 v = {a, b};
    if constexpr (DT == kBF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16_pair));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16_pair));
}

template <int DT>
__device__ __forceinline__ u32x4 narrow16(const float (&v)[Elem<DT>::per16])
{
    if constexpr (DT == kF32)
        return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    else
        return u32x4{narrow2<DT>(v[0], v[1]), narrow2<DT>(v[2], v[3]), narrow2<DT>(v[4], v[5]), narrow2<DT>(v[6], v[7])};
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, size_t i)
{
    if constexpr (DT == kF32) return static_cast<const float*>(p)[i];
    else if constexpr (DT == kBF16) return bf16lo(static_cast<const uint16_t*>(p)[i]);
    else return f16lo(static_cast<const uint16_t*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store1(void* p, size_t i, float v)
{
    if constexpr (DT == kF32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = (uint16_t)narrow2<DT>(v, 0.0f);
}

// Element of a type known at run time (weights: one uniform branch).
__device__ __forceinline__ float load1_rt(const void* p, int dt, size_t i)
{
    return dt == kF32 ? load1<kF32>(p, i) : dt == kBF16 ? load1<kBF16>(p, i) : load1<kF16>(p, i);
}

// Elements [i, end) of a row as a vector of fewer than per16 elements, +0 after.
template <int DT>
__device__ __forceinline__ u32x4 load_tail(const void* row, size_t i, size_t end)
{
    constexpr int E = Elem<DT>::per16, S = Elem<DT>::size;
    const uint8_t* p = static_cast<const uint8_t*>(row) + i * S;
    u32x4 u = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (i + e >= end) continue;
        if constexpr (S == 4) u[e] = reinterpret_cast<const uint32_t*>(p)[e];
        else u[e / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e % 2));
    }
    return u;
}

// N vectors of a row of `end` elements, `step` elements apart from element i
// on; +0 beyond the end.  All whole vectors are asked for before the one that
// the row's end may cut (none where `end` is a multiple of a vector) is read
// by elements, so nothing waits between them.
template <int DT, int N>
__device__ __forceinline__ void load_row(const void* row, size_t i, size_t step, size_t end, u32x4 (&u)[N])
{
    constexpr int E = Elem<DT>::per16, S = Elem<DT>::size;
    const uint8_t* p = static_cast<const uint8_t*>(row);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        u[j] = u32x4{0, 0, 0, 0};
        if (i + j * step + E <= end) u[j] = *reinterpret_cast<const u32x4_any*>(p + (i + j * step) * S);
    }
    if (end % E) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (i + j * step < end && i + j * step + E > end) u[j] = load_tail<DT>(row, i + j * step, end);
    }
}

template <int DT>
__device__ __forceinline__ void store16(void* row, size_t i, size_t end, const u32x4 u)
{
    constexpr int E = Elem<DT>::per16, S = Elem<DT>::size;
    uint8_t* p = static_cast<uint8_t*>(row) + i * S;
    if (i + E <= end) { *reinterpret_cast<u32x4_any*>(p) = u; return; }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (i + e >= end) continue;
        if constexpr (S == 4) reinterpret_cast<uint32_t*>(p)[e] = u[e];
        else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(u[e / 2] >> (16 * (e % 2)));
    }
}

// The value moved by a DPP control within rows of 16 lanes (all lanes active).
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Sum over the 64 lanes, in every lane: pairs, quads, rows of 16 (DPP), then
// the four row sums read out.
__device__ __forceinline__ float wave_total(float v)
{
    v += dpp_move<0xB1>(v);
    v += dpp_move<0x4E>(v);
    v += dpp_move<0x124>(v);
    v += dpp_move<0x128>(v);
    const int i = __float_as_int(v);
    return (__int_as_float(__builtin_amdgcn_readlane(i, 0)) + __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
           (__int_as_float(__builtin_amdgcn_readlane(i, 32)) + __int_as_float(__builtin_amdgcn_readlane(i, 48)));
}

// Sum over a workgroup of W waves, in every lane.  `slot` is LDS of W floats
// that no lane reads between this call's barrier and the next one.
template <int W>
__device__ __forceinline__ float group_total(float v, float* slot)
{
    v = wave_total(v);
    if constexpr (W == 1) return v;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = slot[0];
#pragma unroll
    for (int w = 1; w < W; ++w) s += slot[w];
    return s;
}

}  // namespace rc
