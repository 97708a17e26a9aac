// Products grouped by expert on MXFP4-packed weights, ragged groups of rows.
//
//   forward   y[i][:]  = W_e x[i][:]            off[e] <= i < off[e+1]
//   rows'     dx[i][:] = W_e^T dy[i][:]
//   weights'  dW[e]    = sum over the group's rows of dy[i] x[i]^T
//
// W_e is n x k, row-major, all experts in one packed stream of E n k elements.
// The matrix cores multiply bfloat16: every value that an E2M1 code and an
// E8M0 scale stand for is a bfloat16 (subnormals and overflow to infinity
// included), so weights are decoded without rounding.  Rows in fp16 and fp32
// are cut into P = 2 and 3 bfloat16 terms that add up to them (fp16 exactly,
// fp32 to 2^-24), one product per term; all sums are binary32.
//
// The groups' bounds are read by the kernels: a tile index is mapped to its
// expert by a wave-wide scan of the bounds, and a grid for the largest number
// of tiles that the sizes allow is launched (surplus workgroups end at once).
// Bounds are clamped to the rows there are, so no bounds can reach outside.
#include "rc_op.hpp"
#include "rc_op_launch.hpp"

namespace rc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr size_t kMaxGrid = 0x7FFFFFFF;          // workgroups of a launch

enum : int { kFwd = 0, kDx = 1, kDw = 2 };

template <int DT> struct Terms { static constexpr int v = DT == kBF16 ? 1 : DT == kF16 ? 2 : 3; };

// Rows [lo, hi) of segment s: 0 = rows before the first expert's, 1..E the
// experts, E + 1 = rows after the last one's.
struct Segment { int64_t lo, hi; };
__device__ __forceinline__ Segment segment(const int32_t* off, int experts, int64_t rows, int s)
{
    int64_t lo = s == 0 ? 0 : off[s - 1], hi = s > experts ? rows : off[s];
    lo = lo < 0 ? 0 : lo > rows ? rows : lo;
    hi = hi < lo ? lo : hi > rows ? rows : hi;
    return {lo, hi};
}

// The segment and the first row of row tile `tile` of BM rows; false when
// there are fewer tiles.  Every wave scans for itself: 64 segments at a time.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* off, int experts, int64_t rows, int64_t tile, int& seg,
                                          int64_t& row, int64_t& end)
{
    const int lane = threadIdx.x & 63;
    int64_t before = 0;
    for (int s0 = 0; s0 < experts + 2; s0 += 64) {
        const int s = s0 + lane;
        Segment g = {0, 0};
        if (s < experts + 2) g = segment(off, experts, rows, s);
        const int mine = (int)((g.hi - g.lo + BM - 1) / BM);
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(upto, d, 64);
            if (lane >= d) upto += v;
        }
        const uint64_t past = __builtin_amdgcn_ballot_w64(before + upto > tile);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int64_t first = before + __shfl(upto - mine, l, 64);
            seg = s0 + l;
            row = (int64_t)__shfl(g.lo, l, 64) + (tile - first) * BM;
            end = (int64_t)__shfl(g.hi, l, 64);
            return true;
        }
        before += __shfl(upto, 63, 64);
    }
    return false;
}

// v as P bfloat16 terms, the largest first: each is what is left, rounded
// (cut, where rounding would reach infinity).  An infinity or a NaN is all in
// the first term.
template <int P>
__device__ __forceinline__ void split(float v, uint16_t (&t)[P])
{
#pragma unroll
    for (int p = 0; p < P; ++p) {
        t[p] = (uint16_t)narrow2<kBF16>(v, 0.0f);
        if (p + 1 < P) {
            const bool finite = __builtin_fabsf(v) < __builtin_inff();
            if (finite && (t[p] & 0x7FFF) == 0x7F80) t[p] = (uint16_t)(__float_as_uint(v) >> 16);
            v = finite ? v - __uint_as_float((uint32_t)t[p] << 16) : 0.0f;
        }
    }
}

// ---- the tile kernel ---------------------------------------------------
//
// A BM x BN tile of the result per workgroup of WM x WN waves, BK = 64 of the
// contracted dimension at a time.  Both operands pass through LDS, two buffers
// of each: while the matrix cores work on one, the next step's global loads
// are in flight to registers; they are decoded (weights), cut into terms (fp16
// and fp32 rows) and stored to the other buffer after the products, and one
// barrier ends the step.
//
// An operand lies in LDS as its memory has it: "row" (contraction innermost:
// the rows and, forward, the weights), read with 16-byte loads; or "column"
// (contraction outermost: the weights for dx, both operands of dW), read with
// the transposing loads, which give lane i column i of four rows.  Both are
// swizzled (row_at, col_at) so that the lanes of one load fall on all banks.
//
// The products are formed as weights x rows, so a lane's four results are
// neighbours in the output's row and are stored together.

constexpr int kBK = 64;

// Byte offset of 16-byte unit c (eight contraction values) of row r.
__device__ __forceinline__ uint32_t row_at(uint32_t r, uint32_t c) { return r * (kBK * 2) + ((c ^ (r >> 1 & 7)) << 4); }
// Byte offset of unit c (eight columns) of contraction row r of `cols` columns.
template <int COLS>
__device__ __forceinline__ uint32_t col_at(uint32_t r, uint32_t c)
{
    return r * (COLS * 2) + ((c ^ (((r & 3) << 1 | (r & 8)) & (COLS / 8 - 1))) << 4);
}

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

// The unit's P planes (terms), `plane` bytes apart in LDS.
template <int DT, int P>
__device__ __forceinline__ void store_unit(uint8_t* lds, uint32_t plane, const Unit<DT>& u)
{
    if constexpr (P == 1) {
        *reinterpret_cast<u32x4*>(lds) = u.v[0];
    } else {
        float v[8];
        if constexpr (DT == kF32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u.v[e / 4][e % 4]);
        } else {
            widen8<DT>(u.v[0], v);
        }
        u32x4 t[P];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            uint16_t a[P], b[P];
            split<P>(v[e], a);
            split<P>(v[e + 1], b);
#pragma unroll
            for (int p = 0; p < P; ++p) t[p][e / 2] = (uint32_t)a[p] | (uint32_t)b[p] << 16;
        }
#pragma unroll
        for (int p = 0; p < P; ++p) *reinterpret_cast<u32x4*>(lds + p * plane) = t[p];
    }
}

// One block of 32 weights: its codes and its scale.
struct WeightBlock { u32x4 codes; uint32_t scale; };

__device__ __forceinline__ WeightBlock load_block32(const uint8_t* w, int64_t block, bool in)
{
    WeightBlock b = {};
    if (in) {
        const uint8_t* tile = w + block / 64 * 1088;
        b.codes = *reinterpret_cast<const u32x4*>(tile + block % 64 * 16);
        b.scale = tile[1024 + block % 64];
    }
    return b;
}

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

// Values i .. i + 3 of the output, rounded to its type.
__device__ __forceinline__ void store4(void* out, int ot, size_t i, f32x4 v)
{
    if (ot == kF32) *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i) = v;
    else if (ot == kBF16) *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) = u32x2{narrow2<kBF16>(v[0], v[1]), narrow2<kBF16>(v[2], v[3])};
    else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) = u32x2{narrow2<kF16>(v[0], v[1]), narrow2<kF16>(v[2], v[3])};
}

template <int DIR, int DT> struct Planes {
    // dW in fp16 multiplies fp16 as it is
    static constexpr int a = (DIR == kDw && DT == kF16) ? 1 : Terms<DT>::v, b = DIR == kDw ? a : 1;
};

template <int DIR, int DT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void grouped_tile_kernel(const Grouped a, unsigned cols)
{
    constexpr int T = 64 * WM * WN, PA = Planes<DIR, DT>::a, PB = Planes<DIR, DT>::b;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;                 // a wave's fragments
    constexpr bool F16 = DIR == kDw && DT == kF16;
    constexpr uint32_t A_PLANE = BM * kBK * 2, B_PLANE = BN * kBK * 2;
    constexpr int UA = BM * kBK / 8 / T, UB = BN * kBK / (DIR == kDw ? 8 : 32) / T;   // units, or blocks, of a lane
    static_assert(UA >= 1 && UB >= 1 && UA * 8 * T == BM * kBK, "tile and threads");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr uint32_t BUF = PA * A_PLANE + PB * B_PLANE;

    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave / WN, wn = wave % WN;
    const uint32_t m = lane & 15, q = lane >> 4;
    const int64_t nn = a.n, kk = a.k;
    constexpr int ES = Elem<DT>::size;
    int seg;
    int64_t row, end, depth, m_end;              // the tile's first row, the group's end, the contraction's length
    const int64_t col = (int64_t)(blockIdx.x % cols) * BN, n_end = DIR == kFwd ? nn : kk;
    if constexpr (DIR == kDw) {
        const unsigned rt = (unsigned)((nn + BM - 1) / BM), t = blockIdx.x / cols;
        seg = (int)(t / rt) + 1;
        const Segment g = segment(a.offsets, a.experts, a.rows, seg);
        row = (int64_t)(t % rt) * BM; m_end = nn;
        depth = g.hi - g.lo; end = g.lo;         // `end`: the group's first row
    } else {
        if (!find_tile<BM>(a.offsets, a.experts, a.rows, blockIdx.x / cols, seg, row, end)) return;
        m_end = end;
        depth = (seg == 0 || seg > a.experts) ? 0 : DIR == kFwd ? kk : nn;   // rows of no expert: zeros
    }
    const size_t wbase = (size_t)(seg - 1) * nn * kk;
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM * FN; ++i) acc[i / FN][i % FN] = f32x4{0, 0, 0, 0};

    Unit<DT> ra[UA], rb[DIR == kDw ? UB : 1];
    WeightBlock rw[DIR == kDw ? 1 : UB];
    auto load = [&](int64_t c0) {                // step c0's share of this lane, to registers
#pragma unroll
        for (int i = 0; i < UA; ++i) {
            const uint32_t s = i * T + tid;
            if constexpr (DIR == kDw) {          // dy[end + c0 + r][row + 8 c ..]
                const uint32_t r = s / (BM / 8), c = s % (BM / 8);
                ra[i] = load_unit<DT>(static_cast<const uint8_t*>(a.a) + ((size_t)(end + c0 + r) * nn + row + c * 8) * ES,
                                      c0 + r < depth && row + c * 8 < nn);
            } else {
                const uint32_t r = s / (kBK / 8), c = s % (kBK / 8);
                ra[i] = load_unit<DT>(static_cast<const uint8_t*>(a.a) + ((size_t)(row + r) * depth + c0 + c * 8) * ES,
                                      row + r < m_end && c0 + c * 8 < depth);
            }
        }
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const uint32_t s = i * T + tid;
            if constexpr (DIR == kDw) {          // x[end + c0 + r][col + 8 c ..]
                const uint32_t r = s / (BN / 8), c = s % (BN / 8);
                rb[i] = load_unit<DT>(static_cast<const uint8_t*>(a.b) + ((size_t)(end + c0 + r) * kk + col + c * 8) * ES,
                                      c0 + r < depth && col + c * 8 < kk);
            } else if constexpr (DIR == kFwd) {  // block c of W[col + r], from contraction c0 on
                const uint32_t r = s / (kBK / 32), c = s % (kBK / 32);
                rw[i] = load_block32(a.w, (int64_t)((wbase + (size_t)(col + r) * kk + c0) / 32 + c),
                                     col + r < nn && c0 + c * 32 < kk);
            } else {                             // block c of W[c0 + r], from column col on
                const uint32_t r = s / (BN / 32), c = s % (BN / 32);
                rw[i] = load_block32(a.w, (int64_t)((wbase + (size_t)(c0 + r) * kk + col) / 32 + c),
                                     c0 + r < nn && col + c * 32 < kk);
            }
        }
    };
    auto store = [&](uint8_t* buf) {             // and from there to LDS
#pragma unroll
        for (int i = 0; i < UA; ++i) {
            const uint32_t s = i * T + tid;
            if constexpr (DIR == kDw) store_unit<DT, PA>(buf + col_at<BM>(s / (BM / 8), s % (BM / 8)), A_PLANE, ra[i]);
            else store_unit<DT, PA>(buf + row_at(s / (kBK / 8), s % (kBK / 8)), A_PLANE, ra[i]);
        }
        buf += PA * A_PLANE;
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const uint32_t s = i * T + tid;
            if constexpr (DIR == kDw) {
                store_unit<DT, PB>(buf + col_at<BN>(s / (BN / 8), s % (BN / 8)), B_PLANE, rb[i]);
            } else {
                const float scale = __uint_as_float(rw[i].scale << 23);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t at = DIR == kFwd ? row_at(s / (kBK / 32), s % (kBK / 32) * 4 + e)
                                                    : col_at<BN>(s / (BN / 32), s % (BN / 32) * 4 + e);
                    *reinterpret_cast<u32x4*>(buf + at) = decode8(rw[i].codes[e], scale);
                }
            }
        }
    };
    // fragment addresses: lane (m, q) holds contraction values 8 q .. 8 q + 7 of row or column m
    uint32_t at_row[2], at_col_a[FM], at_col_b[FN];
#pragma unroll
    for (int s = 0; s < 2; ++s) at_row[s] = row_at(m, 4 * s + q);
#pragma unroll
    for (int f = 0; f < FM; ++f)
        if constexpr (DIR == kDw) at_col_a[f] = col_at<BM>(8 * q + m / 4, (wm * (BM / WM) + 16 * f) / 8 + m % 4 / 2) + m % 2 * 8;
#pragma unroll
    for (int f = 0; f < FN; ++f)
        if constexpr (DIR != kFwd) at_col_b[f] = col_at<BN>(8 * q + m / 4, (wn * (BN / WN) + 16 * f) / 8 + m % 4 / 2) + m % 2 * 8;
    auto products = [&](const uint8_t* buf) {
#pragma unroll
        for (int s = 0; s < kBK / 32; ++s) {
#pragma unroll
            for (int pb = 0; pb < PB; ++pb) {
                u32x4 fb[FN];
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    const uint8_t* p = buf + PA * A_PLANE + pb * B_PLANE;
                    if constexpr (DIR == kFwd) fb[f] = *reinterpret_cast<const u32x4*>(p + at_row[s] + (wn * (BN / WN) + 16 * f) * (kBK * 2));
                    else fb[f] = load_columns(p + at_col_b[f] + s * 32 * BN * 2, 4 * BN * 2);
                }
#pragma unroll
                for (int pa = 0; pa < PA; ++pa) {
                    if (pa + pb > 2) continue;   // below 2^-24 of the product
                    u32x4 fa[FM];
#pragma unroll
                    for (int f = 0; f < FM; ++f) {
                        const uint8_t* p = buf + pa * A_PLANE;
                        if constexpr (DIR == kDw) fa[f] = load_columns(p + at_col_a[f] + s * 32 * BM * 2, 4 * BM * 2);
                        else fa[f] = *reinterpret_cast<const u32x4*>(p + at_row[s] + (wm * (BM / WM) + 16 * f) * (kBK * 2));
                    }
#pragma unroll
                    for (int i = 0; i < FM; ++i)
#pragma unroll
                        for (int j = 0; j < FN; ++j) acc[i][j] = mfma<F16>(fb[j], fa[i], acc[i][j]);
                }
            }
        }
    };
    if (depth > 0) {
        load(0);
        store(lds);
        __syncthreads();
        uint32_t cur = 0;
        for (int64_t c0 = 0; c0 < depth; c0 += kBK) {
            const bool more = c0 + kBK < depth;
            if (more) load(c0 + kBK);
            products(lds + cur);
            cur ^= BUF;
            if (more) store(lds + cur);
            __syncthreads();
        }
    }
    const size_t obase = DIR == kDw ? wbase : 0;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t r = row + wm * (BM / WM) + 16 * i + m;
        if (r >= m_end) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int64_t c = col + wn * (BN / WN) + 16 * j + 4 * q;
            if (c < n_end) store4(a.out, a.out_t, obase + (size_t)r * n_end + c, acc[i][j]);
        }
    }
}

template <int DIR, int DT, int BM, int BN, int WM, int WN>
hipError_t launch_tile(const Grouped& a, hipStream_t st)
{
    constexpr size_t bytes = 2 * (size_t)(Planes<DIR, DT>::a * BM + Planes<DIR, DT>::b * BN) * kBK * 2;
    static_assert(bytes <= 160 * 1024, "LDS");
    const size_t cols = ((DIR == kFwd ? a.n : a.k) + BN - 1) / BN;
    const size_t some = a.rows < (size_t)a.experts + 2 ? a.rows : (size_t)a.experts + 2;   // segments that end inside a tile
    const size_t tiles = DIR == kDw ? (size_t)((a.n + BM - 1) / BM) * a.experts : a.rows / BM + some;
    if (tiles > kMaxGrid / cols) return hipErrorInvalidConfiguration;
    const auto kernel = &grouped_tile_kernel<DIR, DT, BM, BN, WM, WN>;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * cols)), dim3(64 * WM * WN), bytes, st, a, (unsigned)cols);
    return hipGetLastError();
}

template <int DIR, int DT>
hipError_t launch_t(const Grouped& a, hipStream_t st)
{
    if constexpr (DT == kF32 && DIR == kDw) return launch_tile<DIR, DT, 128, 64, 2, 2>(a, st);
    else if constexpr (DT == kF32) return launch_tile<DIR, DT, 128, 256, 2, 4>(a, st);
    else if constexpr (DT == kF16 && DIR != kDw) return launch_tile<DIR, DT, 128, 256, 2, 4>(a, st);
    else return launch_tile<DIR, DT, 256, 256, 2, 4>(a, st);
}

template <int DIR>
hipError_t launch_dir(int dt, const Grouped& a, hipStream_t st)
{
    return dt == kF32 ? launch_t<DIR, kF32>(a, st) : dt == kF16 ? launch_t<DIR, kF16>(a, st) : launch_t<DIR, kBF16>(a, st);
}

}  // namespace

hipError_t launch_grouped_forward(int dt, const Grouped& a, hipStream_t st) { return launch_dir<kFwd>(dt, a, st); }
hipError_t launch_grouped_dx(int dt, const Grouped& a, hipStream_t st) { return launch_dir<kDx>(dt, a, st); }
hipError_t launch_grouped_dw(int dt, const Grouped& a, hipStream_t st) { return launch_dir<kDw>(dt, a, st); }

}  // namespace rc
