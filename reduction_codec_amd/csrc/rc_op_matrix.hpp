// rc_op_matrix.hpp -- operands of the matrix instructions, shared by the
// operators that use them: rows cut into bfloat16 terms, MXFP4 codes decoded to
// bfloat16, and columns read from LDS.
#pragma once

#include "rc_op.hpp"

namespace rc {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int DT> struct Terms { static constexpr int v = DT == kBF16 ? 1 : DT == kF16 ? 2 : 3; };

template <int DT> struct Unit { u32x4 v[DT == kF32 ? 2 : 1]; };        // eight values as they lie in memory

template <int DT>
__device__ __forceinline__ Unit<DT> load_unit(const uint8_t* p, bool in)
{
    Unit<DT> u = {};
    if (in) {
        u.v[0] = *reinterpret_cast<const u32x4*>(p);
        if constexpr (DT == kF32) u.v[1] = *reinterpret_cast<const u32x4*>(p + 16);
    }
    return u;
}

// Eight values of a row as P bfloat16 terms that add up to them exactly (fp32
// down to 2^-133): the
// leading eight bits cut off, then (fp32) the next eight rounded, then the rest.
template <int DT, int P>
__device__ __forceinline__ void cut_unit(const Unit<DT>& u, u32x4 (&t)[P])
{
    if constexpr (P == 1) {
        t[0] = u.v[0];
    } else {
        float v[8];
        if constexpr (DT == kF32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u.v[e / 4][e % 4]);
        } else {
            widen8<DT>(u.v[0], v);
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            uint32_t w = __builtin_amdgcn_perm(__float_as_uint(v[e + 1]), __float_as_uint(v[e]), 0x07060302u);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                t[p][e / 2] = w;
                if (p + 1 == P) break;
                v[e] -= bf16lo(w);
                v[e + 1] -= bf16hi(w);
                w = narrow2<kBF16>(v[e], v[e + 1]);
            }
        }
    }
}

// The eight codes of a word as bfloat16, times the scale: exact.
__device__ __forceinline__ u32x4 decode8(uint32_t codes, float s)
{
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3))};
}

template <bool F16>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Eight contraction values of a column: two transposing loads, `next` bytes
// (four contraction rows) apart.
__device__ __forceinline__ u32x4 load_columns(const uint8_t* p, uint32_t next)
{
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + next));
    const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
    return u32x4{x.x, x.y, y.x, y.y};
}

}  // namespace rc
