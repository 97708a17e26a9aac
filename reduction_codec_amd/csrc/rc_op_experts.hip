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
typedef float f32x4 __attribute__((ext_vector_type(4)));

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

// Eight consecutive weights of one block from element i (a multiple of 8) on,
// as four words of bfloat16 pairs.
__device__ __forceinline__ void weights8(const uint8_t* w, size_t i, uint32_t (&v)[4])
{
    const uint8_t* tile = w + i / kTile * 1088;
    const uint32_t in = (uint32_t)(i % kTile);
    const uint32_t codes = *reinterpret_cast<const uint32_t*>(tile + in / 2);
    const float s = __uint_as_float((uint32_t)tile[1024 + in / 32] << 23);
    v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0));
    v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1));
    v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2));
    v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3));
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

// One 64 x 64 tile of the result per workgroup of four waves (each 32 x 32:
// 2 x 2 matrix instructions of 16 x 16 x 32), 32 of the contracted dimension at
// a time through LDS.
template <int DIR, int DT, int OT>
__global__ __launch_bounds__(256) void grouped_tile_kernel(const Grouped a, unsigned cols)
{
    constexpr int P = Terms<DT>::v, PB = DIR == kDw ? P : 1, LD = 40;   // 32 + 8: rows on different banks
    __shared__ __attribute__((aligned(16))) uint16_t la[P][64][LD], lb[PB][64][LD];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t nn = a.n, kk = a.k;
    int seg;
    int64_t row, end, col, depth;                // first row and end of the tile's rows, first column, contraction
    int64_t m_end, n_end;
    if constexpr (DIR == kDw) {
        const unsigned rt = (unsigned)((nn + 63) / 64), t = blockIdx.x / cols;
        seg = (int)(t / rt) + 1;
        const Segment g = segment(a.offsets, a.experts, a.rows, seg);
        row = (int64_t)(t % rt) * 64; m_end = nn;
        col = (int64_t)(blockIdx.x % cols) * 64; n_end = kk;
        depth = g.hi - g.lo; end = g.lo;         // `end`: the group's first row
    } else {
        if (!find_tile<64>(a.offsets, a.experts, a.rows, blockIdx.x / cols, seg, row, end)) return;
        m_end = end;
        col = (int64_t)(blockIdx.x % cols) * 64; n_end = DIR == kFwd ? nn : kk;
        depth = (seg == 0 || seg > a.experts) ? 0 : DIR == kFwd ? kk : nn;   // rows of no expert: zeros
    }
    const size_t wbase = (size_t)(seg - 1) * nn * kk;
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i / 2][i % 2] = f32x4{0, 0, 0, 0};

    for (int64_t c0 = 0; c0 < depth; c0 += 32) {
        // A: 64 x 32, B: 64 x 32, contraction innermost in LDS; eight elements of each per lane
        if constexpr (DIR != kDw) {
            const int i = tid / 4, c = tid % 4 * 8;
            const int64_t ld = DIR == kFwd ? kk : nn;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = row + i < m_end && c0 + c + e < depth;
                uint16_t t[P];
                split<P>(in ? load1<DT>(a.a, (size_t)(row + i) * ld + c0 + c + e) : 0.0f, t);
#pragma unroll
                for (int p = 0; p < P; ++p) la[p][i][c + e] = t[p];
            }
        } else {
            const int c = tid / 8, i = tid % 8 * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint16_t t[P];
                split<P>(row + i + e < m_end && c0 + c < depth ? load1<DT>(a.a, (size_t)(end + c0 + c) * nn + row + i + e) : 0.0f, t);
#pragma unroll
                for (int p = 0; p < P; ++p) la[p][i + e][c] = t[p];
                split<P>(col + i + e < n_end && c0 + c < depth ? load1<DT>(a.b, (size_t)(end + c0 + c) * kk + col + i + e) : 0.0f, t);
#pragma unroll
                for (int p = 0; p < P; ++p) lb[p][i + e][c] = t[p];
            }
        }
        if constexpr (DIR == kFwd) {
            const int j = tid / 4, c = tid % 4 * 8;
            uint32_t v[4] = {0, 0, 0, 0};
            if (col + j < n_end && c0 + c < depth) weights8(a.w, wbase + (size_t)(col + j) * kk + c0 + c, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(&lb[0][j][c + 2 * e]) = v[e];
        } else if constexpr (DIR == kDx) {
            const int c = tid / 8, j = tid % 8 * 8;
            uint32_t v[4] = {0, 0, 0, 0};
            if (col + j < n_end && c0 + c < depth) weights8(a.w, wbase + (size_t)(c0 + c) * kk + col + j, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) lb[0][j + e][c] = (uint16_t)(v[e / 2] >> (16 * (e % 2)));
        }
        __syncthreads();
        const int m = wave / 2 * 32 + lane % 16, q = wave % 2 * 32 + lane % 16, c = lane / 16 * 8;
#pragma unroll
        for (int pa = 0; pa < P; ++pa)
#pragma unroll
            for (int pb = 0; pb < PB; ++pb) {
                if (pa + pb > 2) continue;       // below 2^-24 of the product
                bf16x8 fa[2], fb[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    fa[i] = *reinterpret_cast<const bf16x8*>(&la[pa][m + 16 * i][c]);
                    fb[i] = *reinterpret_cast<const bf16x8*>(&lb[pb][q + 16 * i][c]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i / 2][i % 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i / 2], fb[i % 2], acc[i / 2][i % 2], 0, 0, 0);
            }
        __syncthreads();
    }
    const int64_t ld = DIR == kFwd ? nn : kk;
    const size_t obase = DIR == kDw ? wbase : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t r = row + wave / 2 * 32 + i / 2 * 16 + lane / 16 * 4 + e, q = col + wave % 2 * 32 + i % 2 * 16 + lane % 16;
            if (r < m_end && q < n_end) store1<OT>(a.out, obase + (size_t)r * ld + q, acc[i / 2][i % 2][e]);
        }
}

template <int DIR, int DT, int OT>
hipError_t launch_t(const Grouped& a, hipStream_t st)
{
    const size_t cols = ((DIR == kFwd ? a.n : a.k) + 63) / 64;
    const size_t some = a.rows < (size_t)a.experts + 2 ? a.rows : (size_t)a.experts + 2;   // segments that end inside a tile
    const size_t tiles = DIR == kDw ? (size_t)((a.n + 63) / 64) * a.experts : a.rows / 64 + some;
    if (tiles > kMaxGrid / cols) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((grouped_tile_kernel<DIR, DT, OT>), dim3((unsigned)(tiles * cols)), dim3(256), 0, st, a, (unsigned)cols);
    return hipGetLastError();
}

template <int DIR>
hipError_t launch_dir(int dt, int ot, const Grouped& a, hipStream_t st)
{
#define RC_G(D) (ot == kF32 ? launch_t<DIR, D, kF32>(a, st) : ot == kF16 ? launch_t<DIR, D, kF16>(a, st) : launch_t<DIR, D, kBF16>(a, st))
    return dt == kF32 ? RC_G(kF32) : dt == kF16 ? RC_G(kF16) : RC_G(kBF16);
#undef RC_G
}

}  // namespace

hipError_t launch_grouped_forward(int dt, int ot, const Grouped& a, hipStream_t st) { return launch_dir<kFwd>(dt, ot, a, st); }
hipError_t launch_grouped_dx(int dt, int ot, const Grouped& a, hipStream_t st) { return launch_dir<kDx>(dt, ot, a, st); }
hipError_t launch_grouped_dw(int dt, int ot, const Grouped& a, hipStream_t st) { return launch_dir<kDw>(dt, ot, a, st); }

}  // namespace rc
