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
// are cut into P = 2 and 3 bfloat16 terms that add up to them exactly (fp32 to
// the nearest multiple of 2^-133, bfloat16's smallest), one product per term.
// dW in fp32 leaves out three of nine products, in all up to 2^-22 of the
// whole, where binary32 would round to 2^-24 (with eight of them 16 experts of
// 2048 x 4096 take 965 us for 871 at 512 rows each, 148 for 142 at two), and
// the stated bound of its sums has room for it.  fp16 rows are multiplied as
// they are in dW, and forward where fp16 holds all weights.  All sums are
// binary32.  An infinity cut into terms can come out as NaN (it less itself):
// telling it apart costs 3 % of the time in fp32 and 20 in fp16 (192 rows over
// 32 experts of 2048 x 4096 59 us -> 71).
//
// The groups' bounds are read by the kernels: a tile index is mapped to its
// expert by a wave-wide scan of the bounds, and a grid for the largest number
// of tiles that the sizes allow is launched (surplus workgroups end at once).
// Bounds are clamped to the rows there are, so no bounds can reach outside.
#include <type_traits>
#include "rc_op_matrix.hpp"
#include "rc_op_launch.hpp"
#include "rc_op_rules.hpp"

namespace rc {
namespace {

constexpr size_t kMaxGrid = 0x7FFFFFFF;          // workgroups of a launch

enum : int { kDx = 1, kDw = 2 };

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
            const int64_t first = before + __builtin_amdgcn_readlane(upto - mine, l);
            seg = __builtin_amdgcn_readfirstlane(s0 + l);       // wave-uniform, in scalar registers; rows < 2^31
            row = __builtin_amdgcn_readlane((int)g.lo, l) + (tile - first) * BM;
            end = __builtin_amdgcn_readlane((int)g.hi, l);
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// ---- gradients: the tile kernel ----------------------------------------
//
// A BM x BN tile of the result per workgroup of WM x WN waves, BK of the
// contracted dimension at a time.  Both operands pass through LDS, two buffers
// of each: while the matrix cores work on one, the next step's global loads
// are in flight to registers; they are decoded (weights), cut into terms (fp16
// and fp32 rows) and stored to the other buffer after the products, and one
// barrier ends the step.
//
// An operand lies in LDS as its memory has it: "row" (contraction innermost:
// dy for dx), read with 16-byte loads; or "column" (contraction outermost: the
// weights for dx, both operands of dW, here in fp32), read with the transposing loads, which
// give lane i column i of four rows.  Both are swizzled (row_at, col_at) so
// that the lanes of one load fall on all banks.
//
// The products are formed with the tile's columns as the first operand, so a
// lane's four results are neighbours in the output's row and are stored
// together.

// Byte offset of 16-byte unit c (eight contraction values) of row r; BK = 64.
__device__ __forceinline__ uint32_t row_at(uint32_t r, uint32_t c) { return r * 128 + ((c ^ (r >> 1 & 7)) << 4); }
// Byte offset of unit c (eight columns) of contraction row r of `cols` columns.
template <int COLS>
__device__ __forceinline__ uint32_t col_at(uint32_t r, uint32_t c)
{
    return r * (COLS * 2) + ((c ^ (((r & 3) << 1 | (r & 8)) & (COLS / 8 - 1))) << 4);
}

// col_at for decoded weights.  A lane writes two or four neighbouring units, so eight lanes' first units alone would
// share a half or a quarter of the banks; each group of eight units is shifted within its fours by its number.
template <int COLS>
__device__ __forceinline__ uint32_t weight_at(uint32_t r, uint32_t c) { return col_at<COLS>(r, c ^ (c >> 3 & 3)); }

// The unit's P planes (terms), `plane` bytes apart in LDS.
template <int DT, int P>
__device__ __forceinline__ void store_unit(uint8_t* lds, uint32_t plane, const Unit<DT>& u)
{
    u32x4 t[P];
    cut_unit<DT, P>(u, t);
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<u32x4*>(lds + p * plane) = t[p];
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

// Eight codes as fp16: exact for scales that in_f16() lets through.
__device__ __forceinline__ u32x4 decode8_f16(uint32_t codes, float s)
{
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, 3))};
}

// Whether a block of this scale holds normal fp16 values: 0.5 * 2^e >= 2^-14
// and 6 * 2^e <= 65504.
__device__ __forceinline__ bool in_f16(uint32_t scale) { return scale - 114u <= 26u; }

// Values i .. i + 3 of the output, rounded to its type.
__device__ __forceinline__ void store4(void* out, int ot, size_t i, f32x4 v)
{
    if (ot == kF32) *reinterpret_cast<f32x4*>(static_cast<float*>(out) + i) = v;
    else if (ot == kBF16) *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) = u32x2{narrow2<kBF16>(v[0], v[1]), narrow2<kBF16>(v[2], v[3])};
    else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + i) = u32x2{narrow2<kF16>(v[0], v[1]), narrow2<kF16>(v[2], v[3])};
}

template <int DIR, int DT> struct Planes { static constexpr int a = Terms<DT>::v, b = DIR == kDw ? a : 1; };

// Tile t of a grid whose workgroups go to the eight XCDs in turn: runs of `run`
// neighbours (four row tiles, then the next column) stay on one XCD, whose L2
// then holds what they share, and the runs are dealt to the XCDs in turn, so
// that experts with many rows load all of them alike.
__device__ __forceinline__ uint2 tile_of(unsigned block, unsigned run, unsigned cols)
{
    const unsigned i = block / 8, t = ((i / run) * 8 + block % 8) * run + i % run;
    return {t / (4 * cols) * 4 + t % 4, t / 4 % cols};           // row tile, column
}

template <int DIR, int DT, int BM, int BN, int WM, int WN, int BK = 64, int KS = 1>
__global__ __launch_bounds__(64 * WM * WN * KS) void grouped_tile_kernel(const Grouped a, unsigned cols, unsigned run)
{
    constexpr int T = 64 * WM * WN, PA = Planes<DIR, DT>::a, PB = Planes<DIR, DT>::b;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;                 // a wave's fragments
    constexpr uint32_t A_PLANE = BM * BK * 2, B_PLANE = BN * BK * 2;
    constexpr int NB = BN * BK / (DIR == kDw ? 8 : 32);                  // units, or blocks, of the second operand
    constexpr int UA = BM * BK / 8 / T, UB = (NB + T - 1) / T;          // of a lane
    static_assert(UA >= 1 && (NB < T || NB % T == 0) && UA * 8 * T == BM * BK, "tile and threads");
    static_assert(DIR == kDw || BK == 64, "row operands");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr uint32_t BUF = PA * A_PLANE + PB * B_PLANE;

    // KS groups of waves take every KS-th step each, with buffers of their own, and add up in the end
    const uint32_t part = threadIdx.x / T, tid = threadIdx.x % T, lane = tid & 63, wave = tid >> 6, wm = wave / WN, wn = wave % WN;
    const uint32_t m = lane & 15, q = lane >> 4;
    uint8_t* const own = lds + part * 2 * BUF;
    const int64_t nn = a.n, kk = a.k;
    constexpr int ES = Elem<DT>::size;
    int seg;
    int64_t row, end, depth, m_end;              // the tile's first row, the group's end, the contraction's length
    const uint2 tile = tile_of(blockIdx.x, run, cols);
    const int64_t col = (int64_t)tile.y * BN, n_end = kk;
    if constexpr (DIR == kDw) {
        const unsigned rt = (unsigned)((nn + BM - 1) / BM), t = tile.x;
        seg = (int)(t / rt) + 1;
        if (seg > a.experts) return;
        const Segment g = segment(a.offsets, a.experts, a.rows, seg);
        row = (int64_t)(t % rt) * BM; m_end = nn;
        depth = g.hi - g.lo; end = g.lo;         // `end`: the group's first row
    } else {
        if (!find_tile<BM>(a.offsets, a.experts, a.rows, tile.x, seg, row, end)) return;
        m_end = end;
        depth = (seg == 0 || seg > a.experts) ? 0 : nn;   // rows of no expert: zeros
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
                const uint32_t r = s / (BK / 8), c = s % (BK / 8);
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
            } else {                             // block c of W[c0 + r], from column col on
                const uint32_t r = s / (BN / 32), c = s % (BN / 32);
                rw[i] = load_block32(a.w, (int64_t)((wbase + (size_t)(c0 + r) * kk + col) / 32 + c),
                                     s < NB && c0 + r < nn && col + c * 32 < kk);
            }
        }
    };
    auto store = [&](uint8_t* buf) {             // and from there to LDS
#pragma unroll
        for (int i = 0; i < UA; ++i) {
            const uint32_t s = i * T + tid;
            if constexpr (DIR == kDw) store_unit<DT, PA>(buf + col_at<BM>(s / (BM / 8), s % (BM / 8)), A_PLANE, ra[i]);
            else store_unit<DT, PA>(buf + row_at(s / (BK / 8), s % (BK / 8)), A_PLANE, ra[i]);
        }
        buf += PA * A_PLANE;
#pragma unroll
        for (int i = 0; i < UB; ++i) {
            const uint32_t s = i * T + tid;
            if constexpr (DIR == kDw) {
                store_unit<DT, PB>(buf + col_at<BN>(s / (BN / 8), s % (BN / 8)), B_PLANE, rb[i]);
            } else {
                const float scale = __uint_as_float(rw[i].scale << 23);
                if (s >= NB) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t at = weight_at<BN>(s / (BN / 32), s % (BN / 32) * 4 + e);
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
    for (int f = 0; f < FN; ++f) {
        const uint32_t r = 8 * q + m / 4, c = (wn * (BN / WN) + 16 * f) / 8 + m % 4 / 2;
        at_col_b[f] = (DIR == kDw ? col_at<BN>(r, c) : weight_at<BN>(r, c)) + m % 2 * 8;
    }
    auto products = [&](const uint8_t* buf) {
#pragma unroll
        for (int s = 0; s < BK / 32; ++s) {
#pragma unroll
            for (int pb = 0; pb < PB; ++pb) {
                u32x4 fb[FN];
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                    const uint8_t* p = buf + PA * A_PLANE + pb * B_PLANE;
                    fb[f] = load_columns(p + at_col_b[f] + s * 32 * BN * 2, 4 * BN * 2);
                }
#pragma unroll
                for (int pa = 0; pa < PA; ++pa) {
                    if (pa + pb > 2) continue;   // below 2^-22 of the product
                    u32x4 fa[FM];
#pragma unroll
                    for (int f = 0; f < FM; ++f) {
                        const uint8_t* p = buf + pa * A_PLANE;
                        if constexpr (DIR == kDw) fa[f] = load_columns(p + at_col_a[f] + s * 32 * BM * 2, 4 * BM * 2);
                        else fa[f] = *reinterpret_cast<const u32x4*>(p + at_row[s] + (wm * (BM / WM) + 16 * f) * (BK * 2));
                    }
#pragma unroll
                    for (int i = 0; i < FM; ++i)
#pragma unroll
                        for (int j = 0; j < FN; ++j) acc[i][j] = mfma<false>(fb[j], fa[i], acc[i][j]);
                }
            }
        }
    };
    if (depth > 0) {
        const int64_t c1 = (int64_t)part * BK;   // this group's first step; all groups go as often, some into zeros
        load(c1);
        store(own);
        __syncthreads();
        uint32_t cur = 0;
        for (int64_t c0 = 0; c0 < depth; c0 += BK * KS) {
            const bool more = c0 + BK * KS < depth;
            if (more) load(c0 + c1 + BK * KS);
            products(own + cur);
            cur ^= BUF;
            if (more) store(own + cur);
            __syncthreads();
        }
    }
    if constexpr (KS > 1) {                      // the groups' sums, in their order
        static_assert((KS - 1) * FM * FN * T * 16 <= KS * 2 * BUF, "room for the sums");
        f32x4* sums = reinterpret_cast<f32x4*>(lds);
#pragma unroll
        for (int i = 0; i < FM * FN; ++i)
            if (part > 0) sums[((part - 1) * FM * FN + i) * T + tid] = acc[i / FN][i % FN];
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int i = 0; i < FM * FN; ++i)
#pragma unroll
            for (int p = 0; p < KS - 1; ++p) acc[i / FN][i % FN] += sums[(p * FM * FN + i) * T + tid];
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

// ---- dW in 16-bit types: rows straight to LDS ----------------------------
//
// Both operands are rows as they lie in memory, so they need no registers on
// their way: 32 rows of B columns each go to LDS with the buffer loads that
// write there, into four stages, three of which are in flight while the matrix
// cores work on the fourth.  A B x B tile, swizzled as above (the swizzle
// is in the lanes' memory addresses: LDS is written in lane order).
// Rows past the group's end and columns past the last one lie past the
// descriptors' ends and arrive as zeros.  128 x 128 tiles of four waves where
// large ones are few.
//
// 16 experts of 2048 x 4096 in us, against the kernel above with one step in
// flight: mean 8 rows 99 (104), 64: 113 (127), 512: 222 (257, of which writing
// the 537 MB takes 84 at the rate of a copy), 2048: 524 (656; 1.05 PFLOP/s).
// 256 x 128 tiles, two workgroups per unit: 97, 124, 232, 544; stores past the
// cache 150, 156, 261, 583 (a wave writes 64-byte pieces of 16 rows).

typedef __attribute__((address_space(3))) void lds_void;

template <bool F16, int B>
__global__ __launch_bounds__(2 * B, 2) void grouped_dw_kernel(const Grouped a, unsigned cols, unsigned run)
{
    constexpr int BK = 32, WN = B / 64, FM = B / 32, FN = 4, T = 2 * B;   // waves of B / 2 rows by 64 columns
    constexpr uint32_t kOut = 0xFFFFFF00u, A_BYTES = BK * B * 2, STAGE = 2 * A_BYTES;
    // arrays of their own: the compiler then knows which loads to LDS a read has to wait for
    __shared__ __attribute__((aligned(16))) uint8_t s0[STAGE], s1[STAGE], s2[STAGE], s3[STAGE];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    const uint32_t m = lane & 15, q = lane >> 4;
    const int64_t nn = a.n, kk = a.k;
    const uint2 tile = tile_of(blockIdx.x, run, cols);
    const unsigned rt = (unsigned)((nn + B - 1) / B);
    const int seg = (int)(tile.x / rt) + 1;
    if (seg > a.experts) return;
    const int64_t row = (int64_t)(tile.x % rt) * B, col = (int64_t)tile.y * B;
    const Segment g = segment(a.offsets, a.experts, a.rows, seg);
    const int lo = __builtin_amdgcn_readfirstlane((int)g.lo), depth = __builtin_amdgcn_readfirstlane((int)(g.hi - g.lo));   // rows < 2^31
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM * FN; ++i) acc[i / FN][i % FN] = f32x4{0, 0, 0, 0};

    uint32_t off_a[2], off_b[2];                 // the lane's units of a stage, two of each operand
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t s = i * T + tid, r = s / (B / 8), c = s % (B / 8) ^ ((r & 3) << 1 | (r & 8));
        off_a[i] = row + c * 8 < nn ? (r * (uint32_t)nn + c * 8) * 2 : kOut;
        off_b[i] = col + c * 8 < kk ? (r * (uint32_t)kk + c * 8) * 2 : kOut;
    }
    auto load = [&](uint8_t (&stage)[STAGE], int c0) {
        const int rem = max(min(depth - c0, BK), 0);   // rows of this stage; none: all zeros
        const size_t at = (size_t)lo + c0;
        const Rsrc ra = span_rsrc(a.a, (at * nn + row) * 2, __builtin_amdgcn_readfirstlane(max(rem * (int)nn - (int)row, 0) * 2));
        const Rsrc rb = span_rsrc(a.b, (at * kk + col) * 2, __builtin_amdgcn_readfirstlane(max(rem * (int)kk - (int)col, 0) * 2));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(stage + (i * T + wave * 64) * 16), 16, off_a[i], 0, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(stage + A_BYTES + (i * T + wave * 64) * 16), 16, off_b[i], 0, 0, 0);
        }
    };
    uint32_t at_a[FM], at_b[FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) at_a[f] = col_at<B>(8 * q + m / 4, (wm * (B / 2) + 16 * f) / 8 + m % 4 / 2) + m % 2 * 8;
#pragma unroll
    for (int f = 0; f < FN; ++f) at_b[f] = A_BYTES + col_at<B>(8 * q + m / 4, (wn * 64 + 16 * f) / 8 + m % 4 / 2) + m % 2 * 8;
    // Stage `now` holds step t; `then` was step t - 1's and takes step t + 3.  The wait leaves the 8 loads of steps
    // t + 1 and t + 2 in flight and ends this wave's reads of `then`; past the barrier that holds for all waves.
    auto step = [&](uint8_t (&now)[STAGE], uint8_t (&then)[STAGE], int c0) {
        asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        load(then, c0 + 3 * BK);
        __builtin_amdgcn_sched_barrier(0);
        u32x4 fa[FM], fb[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f) fb[f] = load_columns(now + at_b[f], 4 * B * 2);
#pragma unroll
        for (int f = 0; f < FM; ++f) fa[f] = load_columns(now + at_a[f], 4 * B * 2);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mfma<F16>(fb[j], fa[i], acc[i][j]);
    };
    if (depth > 0) {
        load(s0, 0);
        load(s1, BK);
        load(s2, 2 * BK);
        int c0 = 0;
        for (; c0 + 4 * BK <= depth; c0 += 4 * BK) {       // without exits in between: those would make the compiler wait for more
            step(s0, s3, c0);
            step(s1, s0, c0 + BK);
            step(s2, s1, c0 + 2 * BK);
            step(s3, s2, c0 + 3 * BK);
        }
        if (c0 < depth) step(s0, s3, c0);
        if (c0 + BK < depth) step(s1, s0, c0 + BK);
        if (c0 + 2 * BK < depth) step(s2, s1, c0 + 2 * BK);
        if (c0 + 3 * BK < depth) step(s3, s2, c0 + 3 * BK);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing writes to LDS after the workgroup's end
    }
    const size_t obase = (size_t)(seg - 1) * nn * kk;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t r = row + wm * (B / 2) + 16 * i + m;
        if (r >= nn) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int64_t c = col + wn * 64 + 16 * j + 4 * q;
            if (c < kk) store4(a.out, a.out_t, obase + (size_t)r * kk + c, acc[i][j]);
        }
    }
}

// ---- dx in bf16: dy straight to LDS, weights decoded on their way ---------
//
// A 128 x 256 tile of eight waves, 32 of the contraction at a time.  dy goes to
// LDS with the buffer loads that write there, three of four stages ahead; the
// weights come two steps ahead to registers (half a block a lane), are decoded
// during the step before theirs into one of two buffers, and are read from it
// with the transposing loads.  Rows past the group's end, contraction past n
// and columns past k lie past the descriptors' ends and arrive as zeros.
//
// 16 experts of 2048 x 4096 in us, against 128 x 128 and 256 x 256 tiles of the
// kernel above with one step in flight: mean 256 rows 99 (121), mean 512 166
// (205, 215), mean 2048 530 (684, 642; now 1.04 PFLOP/s).  Without the shifts
// that keep LDS writes of weights and reads of rows free of conflicts 40 % of
// LDS's active time went to them: 171 and 544; in the kernel above fp16 took
// 333 for 312.

__global__ __launch_bounds__(512, 2) void grouped_dx_kernel(const Grouped a, unsigned cols, unsigned run)
{
    constexpr int BM = 128, BN = 256, BK = 32, FM = 4, FN = 4;
    constexpr uint32_t kOut = 0xFFFFFF00u, STAGE = BM * BK * 2, WSTAGE = BK * BN * 2;
    __shared__ __attribute__((aligned(16))) uint8_t s0[STAGE], s1[STAGE], s2[STAGE], s3[STAGE], d0[WSTAGE], d1[WSTAGE];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / 4, wn = wave % 4;
    const uint32_t m = lane & 15, q = lane >> 4;
    const int64_t nn = a.n, kk = a.k;
    const uint2 tile = tile_of(blockIdx.x, run, cols);
    const int64_t col = (int64_t)tile.y * BN;
    int seg;
    int64_t row, end;
    if (!find_tile<BM>(a.offsets, a.experts, a.rows, tile.x, seg, row, end)) return;
    const int depth = (seg == 0 || seg > a.experts) ? 0 : (int)nn;   // rows of no expert: zeros
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM * FN; ++i) acc[i / FN][i % FN] = f32x4{0, 0, 0, 0};

    // dy: unit c of row r, at place c ^ (-(r / 4) % 4) of the row's four: the reads take rows 0 .. 3 and 12 .. 15 of one
    // unit with rows 4 .. 11 of the next, and these fall on all banks
    const uint32_t rows = (uint32_t)(end - row < BM ? end - row : BM), r = tid / 4, c = tid % 4 ^ (-(r >> 2) & 3);
    const Rsrc dr = span_rsrc(a.a, (size_t)row * nn * 2, rows * (uint32_t)nn * 2);
    const uint32_t off_r = r < rows ? (r * (uint32_t)nn + c * 8) * 2 : kOut;
    auto load_rows = [&](uint8_t (&stage)[STAGE], int c0) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(dr, (lds_void*)(stage + wave * 1024), 16,
                                                 c0 + (int)c * 8 < depth && off_r != kOut ? off_r + c0 * 2 : kOut, 0, 0, 0);
    };
    // weights: half h of block b of contraction row wr
    struct Half { u32x2 codes; uint32_t scale; };
    const uint32_t wr = tid / 16, b = tid / 2 % 8, h = tid % 2, blocks = (uint32_t)(kk / 32);
    const uint32_t off_w = col + b * 32 < kk ? wr * blocks + b : kOut;
    auto load_half = [&](Half& w, int c0) {
        const int64_t fb = ((int64_t)(seg - 1) * nn + c0) * blocks + col / 32;
        const Rsrc wd = span_rsrc(a.w, (size_t)(fb >> 6) * 1088, 0x7FFFFFFF);
        const uint32_t at = off_w + (uint32_t)(fb & 63);
        const uint32_t out = off_w == kOut || c0 + (int)wr >= depth ? 0xFFFFFFFFu : 0u;   // past the descriptor's end
        w.codes = __builtin_amdgcn_raw_buffer_load_b64(wd, ((at >> 6) * 1088 + (at & 63) * 16 + h * 8) | out, 0, 0);
        w.scale = __builtin_amdgcn_raw_buffer_load_b8(wd, ((at >> 6) * 1088 + 1024 + (at & 63)) | out, 0, 0);
    };
    auto decode = [&](uint8_t (&buf)[WSTAGE], const Half& w) {
        const float s = __uint_as_float(w.scale << 23);
        *reinterpret_cast<u32x4*>(buf + weight_at<BN>(wr, b * 4 + h * 2)) = decode8(w.codes.x, s);
        *reinterpret_cast<u32x4*>(buf + weight_at<BN>(wr, b * 4 + h * 2 + 1)) = decode8(w.codes.y, s);
    };
    uint32_t at_a = (wm * 64 + m) * 64 + ((q ^ (-(m >> 2) & 3)) << 4), at_b[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) at_b[f] = weight_at<BN>(8 * q + m / 4, (wn * 64 + 16 * f) / 8 + m % 4 / 2) + m % 2 * 8;
    // Step t: `now` and `w` hold its operands.  Three loads are issued a step, dy's first, so past 8 of them dy of
    // step t is there; the barrier also ends all waves' reads of `then` (step t - 1) and of `next`.
    auto step = [&](uint8_t (&now)[STAGE], uint8_t (&then)[STAGE], uint8_t (&w)[WSTAGE], uint8_t (&next)[WSTAGE],
                    Half& ahead, const Half& coming, int c0) {
        asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        load_rows(then, c0 + 3 * BK);
        __builtin_amdgcn_sched_barrier(0);
        load_half(ahead, c0 + 3 * BK);
        __builtin_amdgcn_sched_barrier(0);
        u32x4 fa[FM], fb[FN];
#pragma unroll
        for (int f = 0; f < FN; ++f) fb[f] = load_columns(w + at_b[f], 4 * BN * 2);
#pragma unroll
        for (int f = 0; f < FM; ++f) fa[f] = *reinterpret_cast<const u32x4*>(now + at_a + f * 16 * 64);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mfma<false>(fb[j], fa[i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
        decode(next, coming);
    };
    if (depth > 0) {
        Half w0, w1, w2, w3;
        load_half(w0, 0);
        load_half(w1, BK);
        load_half(w2, 2 * BK);
        __builtin_amdgcn_sched_barrier(0);
        load_rows(s0, 0);
        load_rows(s1, BK);
        load_rows(s2, 2 * BK);
        decode(d0, w0);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the steps count on three loads of each of the last ones
        int c0 = 0;
        for (; c0 + 4 * BK <= depth; c0 += 4 * BK) {
            step(s0, s3, d0, d1, w3, w1, c0);
            step(s1, s0, d1, d0, w0, w2, c0 + BK);
            step(s2, s1, d0, d1, w1, w3, c0 + 2 * BK);
            step(s3, s2, d1, d0, w2, w0, c0 + 3 * BK);
        }
        if (c0 < depth) step(s0, s3, d0, d1, w3, w1, c0);
        if (c0 + BK < depth) step(s1, s0, d1, d0, w0, w2, c0 + BK);
        if (c0 + 2 * BK < depth) step(s2, s1, d0, d1, w1, w3, c0 + 2 * BK);
        if (c0 + 3 * BK < depth) step(s3, s2, d1, d0, w2, w0, c0 + 3 * BK);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing writes to LDS after the workgroup's end
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t o = row + wm * 64 + 16 * i + m;
        if (o >= end) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int64_t k = col + wn * 64 + 16 * j + 4 * q;
            if (k < kk) store4(a.out, a.out_t, (size_t)o * kk + k, acc[i][j]);
        }
    }
}

// ---- few rows per expert ------------------------------------------------
//
// Forward with a handful of rows per expert is bound by the weights' bytes, so
// they go from memory straight to the registers that feed the matrix cores.
// A workgroup forms 16 MF rows by 16 NF columns; its KW waves take every KW-th
// span of 512 of the contracted dimension and add up through LDS in the waves'
// order.  For 16 weight rows, lane (m, q) loads block q of four neighbours (64
// contiguous bytes of a row); one exchange among the four q of a row gives it
// eight codes of each of the four blocks, as the matrix instructions take them
// (contraction values 8 q .. 8 q + 7 of a block), so that the rows' values are
// read 64 contiguous bytes at a time too.

// Word i of lane row q (of 16 lanes) to word q of lane row i.
__device__ __forceinline__ u32x4 exchange(u32x4 c)
{
    const auto a = __builtin_amdgcn_permlane32_swap(c.x, c.z, false, false), b = __builtin_amdgcn_permlane32_swap(c.y, c.w, false, false);
    const auto e = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false), o = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{(uint32_t)e[0], (uint32_t)e[1], (uint32_t)o[0], (uint32_t)o[1]};
}

// v[i] = the value that lane row i holds, in every lane row.
__device__ __forceinline__ void spread(uint32_t x, uint32_t (&v)[4])
{
    const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const auto e = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false), o = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
    v[0] = e[0]; v[1] = e[1]; v[2] = o[0]; v[3] = o[1];
}

template <int DT, int MF, int NF, int KW, bool SPANS>
__global__ __launch_bounds__(64 * KW) void grouped_thin_kernel(const Grouped a, unsigned cols)
{
    constexpr int P = Terms<DT>::v, ES = Elem<DT>::size, RU = DT == kF32 ? 2 : 1;
    constexpr uint32_t kOut = 0xFFFFFF00u;           // past every descriptor's end: reads as zeros, moves nothing
    __shared__ f32x4 part[KW][NF * MF][64];
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, m = lane & 15, q = lane >> 4;
    const int64_t nn = a.n, kk = a.k, col = (int64_t)(blockIdx.x % cols) * (16 * NF);
    const uint32_t blocks = (uint32_t)(kk / 32);
    int seg;
    int64_t row, end;
    if (!find_tile<16 * MF>(a.offsets, a.experts, a.rows, blockIdx.x / cols, seg, row, end)) return;
    const bool none = seg == 0 || seg > a.experts;   // rows of no expert: zeros
    // the workgroup's weight rows and rows, each through one buffer descriptor with 32-bit offsets
    const int64_t fb = ((int64_t)(seg - 1) * nn + col) * blocks;
    const uint32_t wrows = (uint32_t)(nn - col < 16 * NF ? nn - col : 16 * NF), skip = (uint32_t)(fb & 63);
    const uint32_t xrows = (uint32_t)(end - row < 16 * MF ? end - row : 16 * MF);
    const Rsrc wr = span_rsrc(a.w, none ? 0 : (size_t)(fb >> 6) * 1088, none ? 0 : (skip + wrows * blocks + 63) / 64 * 1088);
    const Rsrc xr = span_rsrc(a.a, (size_t)row * kk * ES, xrows * (uint32_t)kk * ES);
    uint32_t first[NF];                              // the lane's weight rows' first blocks
#pragma unroll
    for (int f = 0; f < NF; ++f) first[f] = 16 * f + m < wrows ? skip + (16 * f + m) * blocks : kOut;
    f32x4 acc[NF][MF];
#pragma unroll
    for (int i = 0; i < NF * MF; ++i) acc[i / MF][i % MF] = f32x4{0, 0, 0, 0};

    struct Span { u32x4 codes[NF][4]; uint32_t scale[NF][4]; };
    // blocks b0 + q, + 4, + 8, + 12 of the lane's weight rows (zeros past the row's end)
    auto load_weights = [&](Span& w, uint32_t b0) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            if constexpr (SPANS) {
                const uint32_t at = first[f] + b0;
                const uint32_t tile = (first[f] == kOut || b0 >= blocks) ? kOut : (at >> 6) * 1088, in = at & 63;
                const u32x4 sc = __builtin_amdgcn_raw_buffer_load_b128(wr, tile == kOut ? kOut : tile + 1024 + in, 0, 0);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    w.codes[f][s] = __builtin_amdgcn_raw_buffer_load_b128(wr, tile == kOut ? kOut : tile + (in + q + 4 * s) * 16, 0, 0);
                    w.scale[f][s] = sc[s];
                }
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint32_t b = b0 + q + 4 * s, at = first[f] + b;
                    const bool in = first[f] != kOut && b < blocks;
                    w.codes[f][s] = __builtin_amdgcn_raw_buffer_load_b128(wr, in ? (at >> 6) * 1088 + (at & 63) * 16 : kOut, 0, 0);
                    w.scale[f][s] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(wr, in ? (at >> 6) * 1088 + 1024 + (at & 63) : kOut, 0, 0);
                }
            }
        }
    };
    Unit<DT> u[4][MF][4];
    auto load_rows = [&](uint32_t b0) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = b0 + 4 * s + j, at = ((16 * i + m) * (uint32_t)kk + b * 32 + 8 * q) * ES;
                    const uint32_t off = (16 * i + m < xrows && b < blocks) ? at : kOut;
#pragma unroll
                    for (int h = 0; h < RU; ++h) u[s][i][j].v[h] = __builtin_amdgcn_raw_buffer_load_b128(xr, off + 16 * h, 0, 0);
                }
    };
    auto products = [&](const Span& w) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            u32x4 codes[NF];
            uint32_t scale[NF][4];
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                codes[f] = exchange(w.codes[f][s]);
                if constexpr (SPANS) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) scale[f][j] = w.scale[f][s] >> (8 * j) & 255u;
                } else {
                    spread(w.scale[f][s], scale[f]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 t[MF][P];
#pragma unroll
                for (int i = 0; i < MF; ++i) cut_unit<DT, P>(u[s][i][j], t[i]);
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    const u32x4 v = decode8(codes[f][j], __uint_as_float(scale[f][j] << 23));
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int i = 0; i < MF; ++i) acc[f][i] = mfma<false>(v, t[i][p], acc[f][i]);
                }
            }
        }
    };
    if (!none) {
        Span w;
        for (uint32_t b = wave * 16; b < blocks; b += KW * 16) {
            load_rows(b);
            load_weights(w, b);
            __builtin_amdgcn_sched_barrier(0);       // everything asked for before anything is waited for
            products(w);
        }
    }
#pragma unroll
    for (int i = 0; i < NF * MF; ++i) part[wave][i][lane] = acc[i / MF][i % MF];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NF * MF; i += KW) {
        if (i + wave >= NF * MF) break;
        const int k = i + wave;
        f32x4 v = part[0][k][lane];
#pragma unroll
        for (int w = 1; w < KW; ++w) v += part[w][k][lane];
        const int64_t r = row + k % MF * 16 + m, c = col + k / MF * 16 + 4 * q;
        if (r < end && c < nn) store4(a.out, a.out_t, (size_t)r * nn + c, v);
    }
}

template <int DT, int MF, int NF, int KW>
hipError_t launch_thin(const Grouped& a, hipStream_t st)
{
    const size_t cols = (a.n + 16 * NF - 1) / (16 * NF), some = a.rows < (size_t)a.experts + 2 ? a.rows : (size_t)a.experts + 2;
    const size_t tiles = a.rows / (16 * MF) + some;
    if (tiles > kMaxGrid / cols) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(tiles * cols)), group(64 * KW);
    if (a.k % 512 == 0) hipLaunchKernelGGL((grouped_thin_kernel<DT, MF, NF, KW, true>), grid, group, 0, st, a, (unsigned)cols);
    else hipLaunchKernelGGL((grouped_thin_kernel<DT, MF, NF, KW, false>), grid, group, 0, st, a, (unsigned)cols);
    return hipGetLastError();
}

// ---- some rows per expert -----------------------------------------------
//
// As above, but the waves of a workgroup share their rows: each of WN waves
// forms 16 MF rows by 16 NF columns of its own over the whole contraction, the
// weights straight to registers again, two spans of SB blocks in turn, and the
// rows' spans pass through LDS, cut into terms once for all waves.

// Byte offset of 16-byte unit c of row r in a span of SB blocks of 32.
template <int SB>
__device__ __forceinline__ uint32_t span_at(uint32_t r, uint32_t c) { return r * (SB * 64) + ((c ^ (r & 15)) << 4); }

template <int DT, int MF, int NF, int WN, int SB, bool SPANS>
__global__ __launch_bounds__(64 * WN, 2) void grouped_slim_kernel(const Grouped a, unsigned cols)
{
    constexpr int L = DT == kF32 ? 3 : 1, ES = Elem<DT>::size, RU = DT == kF32 ? 2 : 1, S = SB / 4, T = 64 * WN;
    constexpr uint32_t kOut = 0xFFFFFF00u, PLANE = 16 * MF * SB * 64, BUF = L * PLANE;
    constexpr int UX = 16 * MF * SB * 4 / T;         // 16-byte units of a lane
    static_assert(UX * T == 16 * MF * SB * 4, "units and threads");
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), m = lane & 15, q = lane >> 4;
    const int64_t nn = a.n, kk = a.k, col = (int64_t)(blockIdx.x % cols) * (16 * NF * WN) + wave * (16 * NF);
    const uint32_t blocks = (uint32_t)(kk / 32);
    int seg;
    int64_t row, end;
    if (!find_tile<16 * MF>(a.offsets, a.experts, a.rows, blockIdx.x / cols, seg, row, end)) return;
    const bool none = seg == 0 || seg > a.experts;   // rows of no expert: zeros
    const bool live = col < nn && !none;             // a wave past the last column loads nothing
    const int64_t fb = ((int64_t)(seg - 1) * nn + col) * blocks;
    const uint32_t wrows = live ? (uint32_t)(nn - col < 16 * NF ? nn - col : 16 * NF) : 0, skip = (uint32_t)(fb & 63);
    const uint32_t xrows = (uint32_t)(end - row < 16 * MF ? end - row : 16 * MF);
    const Rsrc wr = span_rsrc(a.w, live ? (size_t)(fb >> 6) * 1088 : 0, live ? (skip + wrows * blocks + 63) / 64 * 1088 : 0);
    const Rsrc xr = span_rsrc(a.a, (size_t)row * kk * ES, xrows * (uint32_t)kk * ES);
    uint32_t first[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) first[f] = 16 * f + m < wrows ? skip + (16 * f + m) * blocks : kOut;
    f32x4 acc[NF][MF];
#pragma unroll
    for (int i = 0; i < NF * MF; ++i) acc[i / MF][i % MF] = f32x4{0, 0, 0, 0};

    struct Span { u32x4 codes[NF][S]; uint32_t scale[NF][S]; };
    auto load_weights = [&](Span& w, uint32_t b0) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            if constexpr (SPANS) {
                const uint32_t at = first[f] + b0;
                const uint32_t tile = (first[f] == kOut || b0 >= blocks) ? kOut : (at >> 6) * 1088, in = at & 63;
                if constexpr (S == 4) {
                    const u32x4 sc = __builtin_amdgcn_raw_buffer_load_b128(wr, tile == kOut ? kOut : tile + 1024 + in, 0, 0);
#pragma unroll
                    for (int s = 0; s < S; ++s) w.scale[f][s] = sc[s];
                } else if constexpr (S == 1) {
                    w.scale[f][0] = __builtin_amdgcn_raw_buffer_load_b32(wr, tile == kOut ? kOut : tile + 1024 + in, 0, 0);
                } else {
                    const u32x2 sc = __builtin_amdgcn_raw_buffer_load_b64(wr, tile == kOut ? kOut : tile + 1024 + in, 0, 0);
#pragma unroll
                    for (int s = 0; s < S; ++s) w.scale[f][s] = sc[s];
                }
#pragma unroll
                for (int s = 0; s < S; ++s)
                    w.codes[f][s] = __builtin_amdgcn_raw_buffer_load_b128(wr, tile == kOut ? kOut : tile + (in + q + 4 * s) * 16, 0, 0);
            } else {
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const uint32_t b = b0 + q + 4 * s, at = first[f] + b;
                    const bool in = first[f] != kOut && b < blocks;
                    w.codes[f][s] = __builtin_amdgcn_raw_buffer_load_b128(wr, in ? (at >> 6) * 1088 + (at & 63) * 16 : kOut, 0, 0);
                    w.scale[f][s] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(wr, in ? (at >> 6) * 1088 + 1024 + (at & 63) : kOut, 0, 0);
                }
            }
        }
    };
    Unit<DT> u[UX];
    auto load_rows = [&](uint32_t b0) {              // this lane's units of the rows' span, to registers
#pragma unroll
        for (int i = 0; i < UX; ++i) {
            const uint32_t s = i * T + tid, r = s / (SB * 4), c = s % (SB * 4);
            const uint32_t off = (r < xrows && b0 + c / 4 < blocks) ? (r * (uint32_t)kk + b0 * 32 + c * 8) * ES : kOut;
#pragma unroll
            for (int h = 0; h < RU; ++h) u[i].v[h] = __builtin_amdgcn_raw_buffer_load_b128(xr, off + 16 * h, 0, 0);
        }
    };
    auto store_rows = [&](uint8_t* buf) {            // and from there, as terms, to LDS
#pragma unroll
        for (int i = 0; i < UX; ++i) {
            const uint32_t s = i * T + tid;
            u32x4 t[L];
            cut_unit<DT, L>(u[i], t);
#pragma unroll
            for (int p = 0; p < L; ++p) *reinterpret_cast<u32x4*>(buf + p * PLANE + span_at<SB>(s / (SB * 4), s % (SB * 4))) = t[p];
        }
    };
    auto products = [&](const Span& w, const uint8_t* buf, auto as_f16) {
        constexpr bool F16 = decltype(as_f16)::value;
        constexpr int P = F16 ? 1 : Terms<DT>::v;
        // one step is 32 of the contraction; in large tiles its successor's fragments are read and decoded during
        // its products (the registers would halve the waves of smaller ones)
        constexpr int AHEAD = MF * NF >= 16 && P == L ? 1 : 0, SETS = AHEAD + 1;
        u32x4 t[SETS][MF][P], v[SETS][NF], codes[NF];
        uint32_t scale[NF][4];
        auto fetch = [&](int step) {
            const int s = step / 4, j = step % 4;
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                const uint8_t* at = buf + span_at<SB>(16 * i + m, 4 * step + q);
                if constexpr (L == P) {
#pragma unroll
                    for (int p = 0; p < P; ++p) t[step % SETS][i][p] = *reinterpret_cast<const u32x4*>(at + p * PLANE);
                } else {
                    cut_unit<DT, P>(Unit<DT>{*reinterpret_cast<const u32x4*>(at)}, t[step % SETS][i]);
                }
            }
            if (j == 0) {
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    codes[f] = exchange(w.codes[f][s]);
                    if constexpr (SPANS) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) scale[f][k] = w.scale[f][s] >> (8 * k) & 255u;
                    } else {
                        spread(w.scale[f][s], scale[f]);
                    }
                }
            }
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const float two_e = __uint_as_float(scale[f][j] << 23);
                v[step % SETS][f] = F16 ? decode8_f16(codes[f][j], two_e) : decode8(codes[f][j], two_e);
            }
        };
        if (AHEAD) fetch(0);
#pragma unroll
        for (int step = 0; step < 4 * S; ++step) {
            if (step + AHEAD < 4 * S) fetch(step + AHEAD);
#pragma unroll
            for (int f = 0; f < NF; ++f)
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int i = 0; i < MF; ++i) acc[f][i] = mfma<F16>(v[step % SETS][f], t[step % SETS][i][p], acc[f][i]);
        }
    };
    // the rows' next span is asked for before the next weights, so it can be stored while those are in flight
    auto run = [&](auto as_f16) {
        Span w0, w1;
        load_rows(0);
        load_weights(w0, 0);
        store_rows(lds);
        __syncthreads();
        for (uint32_t b = 0; b < blocks; b += 2 * SB) {
            load_rows(b + SB);
            load_weights(w1, b + SB);
            __builtin_amdgcn_sched_barrier(0);
            products(w0, lds, as_f16);
            store_rows(lds + BUF);
            __syncthreads();
            load_rows(b + 2 * SB);
            load_weights(w0, b + 2 * SB);
            __builtin_amdgcn_sched_barrier(0);
            products(w1, lds + BUF, as_f16);
            store_rows(lds);
            __syncthreads();
        }
    };
    if constexpr (DT == kF16 && MF > 1) {
        if (!none) {
            // fp16 rows are multiplied as they are, once, where fp16 holds all of the workgroup's weights: the scales of
            // their blocks are looked at (16 tiles at a time, 16 bytes a lane), and the codes of a block whose scale is
            // out of fp16's range, for zeros are held whatever it is (the packer gives blocks of zeros the scale
            // 2^-127: with 2 % of them 2331 rows of 1000 x 2080 over 12 experts take 31 us, as two terms 63; 16384 rows
            // of 8192 x 4096 over 8 1.12 ms and 3.10).  Not with few rows, where the weights' bytes count and not the
            // products (192 rows: 39 us, 45 with the look).
            __shared__ uint32_t odd;
            if (tid == 0) odd = 0;
            __syncthreads();
            bool fits = true;
            const uint32_t past = skip + wrows * blocks, tiles = live ? (past + 63) / 64 : 0;
            for (uint32_t i = lane / 4; i < tiles; i += 16) {
                const uint32_t b0 = i * 64 + lane % 4 * 16;
                const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(wr, i * 1088 + 1024 + lane % 4 * 16, 0, 0);
                uint32_t look = 0, nan = 0;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t scale = x[e / 4] >> (8 * (e % 4)) & 255u;
                    look |= (uint32_t)!in_f16(scale) << e;
                    nan |= (uint32_t)(scale == 255u) << e;
                }
                uint32_t mine = 0xFFFFu;             // neighbours' blocks and the stream's padding do not count
                if (b0 < skip) mine &= 0xFFFFu << min(skip - b0, 16u);
                if (b0 + 16 > past) mine &= 0xFFFFu >> min(b0 + 16 - past, 16u);
                fits = fits && (nan & mine) == 0;
                for (look &= mine; look; look &= look - 1) {
                    const u32x4 c = __builtin_amdgcn_raw_buffer_load_b128(wr, i * 1088 + (lane % 4 * 16 + __builtin_ctz(look)) * 16, 0, 0);
                    fits = fits && ((c.x | c.y | c.z | c.w) & 0x77777777u) == 0;
                }
            }
            if (!fits) odd = 1;
            __syncthreads();
            if (odd) run(std::false_type{});
            else run(std::true_type{});
        }
    } else {
        if (!none) run(std::false_type{});
    }
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const int64_t r = row + 16 * i + m, c = col + 16 * f + 4 * q;
            if (r < end && c < nn) store4(a.out, a.out_t, (size_t)r * nn + c, acc[f][i]);
        }
}

template <int DT, int MF, int NF, int WN, int SB>
hipError_t launch_slim(const Grouped& a, hipStream_t st)
{
    constexpr size_t bytes = 2 * (size_t)(DT == kF32 ? 3 : 1) * 16 * MF * SB * 64;
    static_assert(bytes <= 160 * 1024, "LDS");
    const size_t cols = (a.n + 16 * NF * WN - 1) / (16 * NF * WN), some = a.rows < (size_t)a.experts + 2 ? a.rows : (size_t)a.experts + 2;
    const size_t tiles = a.rows / (16 * MF) + some;
    if (tiles > kMaxGrid / cols) return hipErrorInvalidConfiguration;
    const auto kernel = a.k % (SB * 32) == 0 ? &grouped_slim_kernel<DT, MF, NF, WN, SB, true> : &grouped_slim_kernel<DT, MF, NF, WN, SB, false>;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * cols)), dim3(64 * WN), bytes, st, a, (unsigned)cols);
    return hipGetLastError();
}

// Workgroups for `tiles` row tiles by `cols` columns and the runs of tile_of;
// 0 when they are too many.  Runs of 32 tiles where every XCD gets several.
inline size_t tile_grid(size_t tiles, size_t cols, unsigned& run)
{
    if (tiles > (kMaxGrid - 8192) / cols / 4) return 0;
    const size_t total = (tiles + 3) / 4 * 4 * cols;
    run = total >= 1024 ? 32 : total >= 256 ? 4 : 1;
    return (total + 8 * run - 1) / (8 * run) * (8 * run);
}

template <int DIR, int DT, int BM, int BN, int WM, int WN, int BK = 64, int KS = 1>
hipError_t launch_tile(const Grouped& a, hipStream_t st)
{
    constexpr size_t bytes = KS * 2 * (size_t)(Planes<DIR, DT>::a * BM + Planes<DIR, DT>::b * BN) * BK * 2;
    static_assert(bytes <= 160 * 1024, "LDS");
    const size_t cols = (a.k + BN - 1) / BN;
    const size_t some = a.rows < (size_t)a.experts + 2 ? a.rows : (size_t)a.experts + 2;   // segments that end inside a tile
    const size_t tiles = DIR == kDw ? (size_t)((a.n + BM - 1) / BM) * a.experts : a.rows / BM + some;
    unsigned run;
    const size_t grid = tile_grid(tiles, cols, run);
    if (grid == 0) return hipErrorInvalidConfiguration;
    const auto kernel = &grouped_tile_kernel<DIR, DT, BM, BN, WM, WN, BK, KS>;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(64 * WM * WN * KS), bytes, st, a, (unsigned)cols, run);
    return hipGetLastError();
}

template <bool F16, int B>
hipError_t launch_dw(const Grouped& a, hipStream_t st)
{
    const size_t cols = (a.k + B - 1) / B, tiles = (size_t)((a.n + B - 1) / B) * a.experts;
    unsigned run;
    const size_t grid = tile_grid(tiles, cols, run);
    if (grid == 0) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((grouped_dw_kernel<F16, B>), dim3((unsigned)grid), dim3(2 * B), 0, st, a, (unsigned)cols, run);
    return hipGetLastError();
}

hipError_t launch_dx(const Grouped& a, hipStream_t st)
{
    const size_t cols = (a.k + 255) / 256, some = a.rows < (size_t)a.experts + 2 ? a.rows : (size_t)a.experts + 2;
    unsigned run;
    const size_t grid = tile_grid(a.rows / 128 + some, cols, run);
    if (grid == 0) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(grouped_dx_kernel, dim3((unsigned)grid), dim3(512), 0, st, a, (unsigned)cols, run);
    return hipGetLastError();
}

inline GroupedSizes sizes_of(const Grouped& a) { return {a.rows, (size_t)a.experts, a.n, a.k}; }

template <int DT>
hipError_t launch_forward(const Grouped& a, hipStream_t st)
{
    const Forward form = forward_form(DT == kF32, sizes_of(a));
    if (form == Forward::kThin16x32) return launch_thin<DT, 1, 2, 4>(a, st);
    if (form == Forward::k16x128) return launch_slim<DT, 1, 1, 8, DT == kF32 ? 8 : 16>(a, st);
    if constexpr (DT == kF32) {
        if (form == Forward::k32x128F32) return launch_slim<DT, 2, 2, 4, 4>(a, st);
        return launch_slim<DT, 2, 2, 8, 4>(a, st);
    } else {
        switch (form) {
        case Forward::k32x128Span16: return launch_slim<DT, 2, 1, 8, 16>(a, st);
        case Forward::k32x128Span8: return launch_slim<DT, 2, 1, 8, 8>(a, st);
        case Forward::k64x128: return launch_slim<DT, 4, 1, 8, 8>(a, st);
        case Forward::k64x256: return launch_slim<DT, 4, 2, 8, 4>(a, st);
        case Forward::k128x128: return launch_slim<DT, 8, 2, 4, 4>(a, st);
        default: return launch_slim<DT, 8, 2, 8, 4>(a, st);
        }
    }
}

template <int DIR, int DT>
hipError_t launch_backward(const Grouped& a, hipStream_t st)
{
    if constexpr (DIR == kDx) {
        const Dx form = dx_form(DT == kBF16, sizes_of(a));
        if (form == Dx::k64x64Shared) return launch_tile<DIR, DT, 64, 64, 2, 2, 64, DT == kBF16 ? 4 : 2>(a, st);
        if (form == Dx::k64x128) return launch_tile<DIR, DT, 64, 128, 2, 2>(a, st);
        if constexpr (DT == kBF16) return launch_dx(a, st);
        else return launch_tile<DIR, DT, 128, 256, 2, 4>(a, st);
    } else if constexpr (DT == kF32) {
        return launch_tile<DIR, DT, 128, 128, 2, 4, 32>(a, st);
    } else {
        return dw_form(false, sizes_of(a)) == Dw::k128x128 ? launch_dw<DT == kF16, 128>(a, st) : launch_dw<DT == kF16, 256>(a, st);
    }
}

template <int DIR>
hipError_t launch_backward_rt(int dt, const Grouped& a, hipStream_t st)
{
    return dt == kF32 ? launch_backward<DIR, kF32>(a, st) : dt == kF16 ? launch_backward<DIR, kF16>(a, st) : launch_backward<DIR, kBF16>(a, st);
}

}  // namespace

hipError_t launch_grouped_forward(int dt, const Grouped& a, hipStream_t st)
{
    return dt == kF32 ? launch_forward<kF32>(a, st) : dt == kF16 ? launch_forward<kF16>(a, st) : launch_forward<kBF16>(a, st);
}

hipError_t launch_grouped_dx(int dt, const Grouped& a, hipStream_t st) { return launch_backward_rt<kDx>(dt, a, st); }
hipError_t launch_grouped_dw(int dt, const Grouped& a, hipStream_t st) { return launch_backward_rt<kDw>(dt, a, st); }

}  // namespace rc
