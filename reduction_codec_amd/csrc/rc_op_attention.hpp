// Attention over a paged cache held in MXFP4: the kernels, instantiated per
// type of the queries in the rc_op_attention_*.hip units.
//
//   s_j = scale q . K_j,  out = sum exp(s_j - m) V_j / sum exp(s_j - m),
//   lse = m + log sum exp(s_j - m),  m = max s_j
//
// One pass over the tokens with a running maximum.  Everything is computed
// transposed, S^T = K Q^T and out^T = V^T P^T, sixteen tokens by sixteen rows of
// q at a time: a lane then holds scores of four tokens and one row, which are
// the second operand of the second product as they stand (what order the
// contraction takes its 32 tokens in is free, as long as V follows), and a row's
// maximum and sum are a lane's own but for four lanes that meet at the end.
//
// The rows of a sequence are its tokens times the heads that share a head of
// the cache.  What an E2M1 code under an E8M0 scale stands for is a bfloat16, so
// keys and values are decoded exactly; queries are cut into one (bf16), two
// (fp16) or three (fp32) bfloat16 terms that add up to them, and so are the
// weights exp(s_j - m).  One term rounds them to half a step of bfloat16, 2^-8 at
// most of themselves: bf16 results, whose own rounding is as large, are then off by
// 0.0021 of their norm (normal values), 0.0016 with a second term.  That would cost more than it
// gives where the matrix cores bound (us with one and two: prompts of 4500 tokens on
// average 468, 549; chunks behind 30000 359, 439; heads of 256 1038, 1196).
#pragma once

#include "rc_op_cache.hpp"
#include "rc_op_matrix.hpp"
#include "rc_op_rules.hpp"

namespace rc {

constexpr int kRowWaves = 4;                     // of a workgroup
constexpr int kUnit = 32 * kRowWaves;            // tokens of a unit of work

// ---- a row of D = 32 NB values over four lanes
//
// Four lanes g hold the NB 4-byte words (eight codes each) of a token's row that
// the NB matrix instructions of a score take: four blocks at a time a block each
// (16 bytes), then two blocks as halves, then one as quarters.
template <int NB>
struct RowMap {
    static constexpr int kFours = NB / 4, kPieces = NB / 4 + (NB % 4 >= 2) + NB % 2;
    // words of piece p: the first one's number (and first block's) and how many a lane has
    static constexpr int first(int p) { return p < kFours ? 4 * p : p == kFours && NB % 4 >= 2 ? 4 * kFours : NB - 1; }
    static constexpr int words(int p) { return p < kFours ? 4 : p == kFours && NB % 4 >= 2 ? 2 : 1; }
    static constexpr int piece(int s) { return s < 4 * kFours ? s / 4 : NB % 4 == 1 ? kFours : s - 4 * kFours < 2 ? kFours : kFours + 1; }
    // block of lane g's words of piece p, and their byte in it
    static __device__ __forceinline__ uint32_t block(int p, uint32_t g)
    {
        return first(p) + (words(p) == 4 ? g : words(p) == 2 ? g / 2 : 0);
    }
    static __device__ __forceinline__ uint32_t byte(int p, uint32_t g)
    {
        return words(p) == 4 ? 0 : words(p) == 2 ? g % 2 * 8 : g * 4;
    }
    // the eight values of lane g's word s: 8 unit(s, g) ..
    static __device__ __forceinline__ uint32_t unit(int s, uint32_t g)
    {
        return block(piece(s), g) * 4 + byte(piece(s), g) / 4 + (s - first(piece(s)));
    }
};

// ---- 32 tokens' codes
//
// They are asked for in the order of memory, a lane a block (16 bytes, kLoads
// times): lanes that took their words as the matrix instructions want them, 64
// bytes apart, would touch four times the lines (64 long sequences, bf16, heads of
// 128: 87 us for loads from the first cache alone).  Keys are handed to the lanes
// that multiply them through LDS, as they are; values pass through LDS anyway.
// Scales come as words that hold them (a byte's load would be widened as soon as
// it is there, and so waited for): of keys for the lane that multiplies, of
// values for the lane that has the block.
template <int NB> constexpr int kLoads = (NB + 1) / 2;
template <int NB> constexpr bool kHalves = NB % 4 == 0;  // sixteen tokens are whole tiles, and each sixteen may have a page of its own

template <int NB>
struct Codes {
    u32x4 w[kLoads<NB>];
};

// Where sixteen tokens' codes lie in the cache: the byte of the tile that they
// begin in, and, below its 16, how many sixteens of blocks into it (of 64, 96 and
// 192 values sixteen tokens are no whole tiles) and whether there is no such page.
constexpr uint32_t kNoPage = 4;
template <int NB>
__device__ __forceinline__ uint64_t group_at(const Cache& c, int page, int head, uint32_t k16)
{
    if (page < 0 || page >= c.pages) return kNoPage;
    const uint32_t b0 = 16 * NB * k16;
    return stream_at(c, page, head) + b0 / 64 * kMxTile + b0 % 64 / 16;
}
__device__ __forceinline__ const uint8_t* tile_at(const uint8_t* cache, uint64_t where) { return cache + (where & ~(uint64_t)15); }
__device__ __forceinline__ uint32_t block_in(uint64_t where) { return ((uint32_t)where & 3) * 16; }

// Lane's block of load j, among the 32 NB of the tokens (a lane beyond them has its first again).
template <int NB>
__device__ __forceinline__ uint32_t block_of(int j, uint32_t lane)
{
    const uint32_t b = 64 * j + lane;
    return b < 32 * NB ? b : lane;
}

// The tile and the block in it of load j's block b: the tokens of a page lie
// together, from its first sixteen on; where tiles are whole each sixteen counts for itself.
template <int NB>
struct Spot {
    const uint8_t* tile;
    uint32_t block;
};
template <int NB>
__device__ __forceinline__ Spot<NB> spot_of(const uint8_t* cache, const uint64_t (&where)[2], int j, uint32_t b)
{
    if constexpr (kHalves<NB>) return {tile_at(cache, where[j / (NB / 4)]), b - j / (NB / 4) * (16 * NB)};
    else return {tile_at(cache, where[0]), block_in(where[0]) + b};
}

template <int NB>
__device__ __forceinline__ void load_codes(const uint8_t* cache, const uint64_t (&where)[2], uint32_t lane, Codes<NB>& c)
{
#pragma unroll
    for (int j = 0; j < kLoads<NB>; ++j) {
        const Spot<NB> p = spot_of<NB>(cache, where, j, block_of<NB>(j, lane));
        c.w[j] = *reinterpret_cast<const u32x4*>(p.tile + codes_at(p.block));
    }
}

// The word that holds the scale of block b of a tile's stream, and the scale in it.
__device__ __forceinline__ uint32_t load_scale(const uint8_t* tile, uint32_t b) { return *reinterpret_cast<const uint32_t*>(tile + (scale_at(b) & ~3u)); }
__device__ __forceinline__ uint32_t scale_byte(uint32_t word, uint32_t b) { return __builtin_amdgcn_ubfe(word, b % 4 * 8, 8); }
__device__ __forceinline__ float scale_of(uint32_t word, uint32_t b) { return __uint_as_float(scale_byte(word, b) << 23); }

// Whether a block of four words and this scale has values that binary32 does not
// hold: all of NaN, 2 and more under 2^127, 4 and more under 2^126 (bit 2 of a code
// says 2 or more, with bit 1 4 or more).
__device__ __forceinline__ bool not_finite(u32x4 w, uint32_t scale)
{
    const uint32_t two = w.x | w.y | w.z | w.w, four = (w.x & w.x << 1) | (w.y & w.y << 1) | (w.z & w.z << 1) | (w.w & w.w << 1);
    return scale >= 253 && (scale == 255 || ((scale == 254 ? two : four) & 0x44444444u) != 0);
}

// Keys' codes in LDS: a token's blocks, and an odd number of 16-byte units from
// one token to the next, so that eight tokens' fall on all banks.
template <int NB> constexpr uint32_t kKeyRow = (NB | 1) * 16;

// ---- values in LDS: rows of D bfloat16 values, one a token, 32 bytes apart: the
// sixteen lanes of a step of a transposing load (four tokens, two 16-byte units)
// then fall on all banks (D / 8 + 2 units are 2 modulo 8, or 6).  So do the eight
// lanes of a step of a store, of one or more tokens' blocks (four units each),
// if neighbouring pairs of blocks begin with different units of their four.
template <int NB>
__device__ __forceinline__ u32x4 turned(u32x4 w, uint32_t by)
{
    if (NB > 4) w = by & 2 ? u32x4{w.z, w.w, w.x, w.y} : w;
    return by & 1 ? u32x4{w.y, w.z, w.w, w.x} : w;
}
template <int NB> constexpr uint32_t kValueRow = NB * 64 + 32;
template <int NB>
__device__ __forceinline__ uint32_t value_at(uint32_t token, uint32_t unit)
{
    return token * kValueRow<NB> + unit * 16;
}

// Largest over the four lanes that share a row, in each of them.
__device__ __forceinline__ float max_of_row(float v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
// Sum over the four lanes that share a row, in each of them.
__device__ __forceinline__ float sum_of_row(float v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// Weights of 2 x 4 tokens as P bfloat16 terms that add up to them (to 2^-8,
// 2^-17 and 2^-24 of themselves).
template <int P>
__device__ __forceinline__ void cut_weights(const float (&p)[8], u32x4 (&t)[P])
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = p[e];
#pragma unroll
    for (int x = 0; x < P; ++x)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint32_t w = narrow2<kBF16>(v[e], v[e + 1]);
            t[x][e / 2] = w;
            v[e] -= bf16lo(w);
            v[e + 1] -= bf16hi(w);
        }
}

// What lanes of a wave write to LDS, others read: the order is the hardware's
// own, the compiler must keep it.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// ---- work
//
// A sequence's rows are cut into tiles of R.  A tile has units of 128 tokens, as
// many as its rows see; the first tile of a causal sequence sees the fewest and
// the last the most, so tile j and the j-th from the end go together as a pair,
// and all pairs of a sequence count alike (a pair may end in units that stand
// for nothing).  All units of all pairs of all sequences stand in one row, which
// is cut into ranges of one length, so that sequences of all lengths load the card
// alike, and a workgroup takes a range of one head.  The workgroups of the heads
// of a range run side by side: what they read of a page lies together (64 long
// sequences, bf16, heads of 128: 4.6 TB/s where heads followed one another, 5.0
// so).  A tile that is cut is joined by a second kernel: a workgroup leaves at most
// two parts, of the tile that it takes over (slot 2 w) and of the one that it
// leaves (slot 2 w + 1).
struct Sequence {
    int row0, tokens, length;                    // first row of q; rows; tokens in the cache
};

// Tiles of a sequence, and units of a pair of them (of the only one).
struct Tiles {
    int tiles, pairs;
    int64_t units;                               // of a pair
};

// What the tile's rows see: the first token (a multiple of 32), and its units.
struct Extent {
    int first, units;
};

// The tokens that row r sees: lo <= j < hi.
__device__ __forceinline__ void row_sees(const CacheAttention& a, const Sequence& q, uint32_t group, uint32_t r, int& lo, int& hi)
{
    const int64_t p = (int64_t)q.length - q.tokens + r / group;
    hi = a.causal ? (p < q.length ? (int)(p + 1 < 0 ? 0 : p + 1) : q.length) : q.length;
    lo = a.window != 0 && p - a.window + 1 > 0 ? (int)(p - a.window + 1) : 0;
}

template <int R>
__device__ __forceinline__ Extent extent(const CacheAttention& a, const Sequence& q, uint32_t group, int tile)
{
    const uint32_t rows = (uint32_t)q.tokens * group, r0 = (uint32_t)tile * R, r1 = rows - r0 < R ? rows : r0 + R;
    int lo, hi, none;
    row_sees(a, q, group, r0, lo, none);
    row_sees(a, q, group, r1 - 1, none, hi);
    lo &= ~31;
    return {lo, hi > lo ? (hi - lo + kUnit - 1) / kUnit : 1};        // rows that see nothing are written all the same
}

template <int R>
__device__ __forceinline__ Tiles tiles_of(const CacheAttention& a, const Sequence& q, uint32_t group)
{
    if (q.tokens == 0) return {0, 0, 0};
    const int n = (int)(((uint32_t)q.tokens * group + R - 1) / R);
    if (n == 1) return {1, 1, extent<R>(a, q, group, 0).units};
    const int64_t whole = q.length > 0 ? ((int64_t)q.length + kUnit - 1) / kUnit : 1;
    int64_t u = 2 * whole;
    const int64_t before = (int64_t)q.length - q.tokens;
    if (a.causal && before >= 0) {               // both ends' last rows, rounded up to units
        const int64_t v = (2 * (before + 1) + ((int64_t)n + 1) * R / group) / kUnit + 2;
        u = v < u ? v : u;
    }
    if (a.window != 0) {
        const int64_t v = 2 * (((int64_t)a.window + R / group + 33) / kUnit + 2);
        u = v < u ? v : u;
    }
    return {n, (n + 1) / 2, u};
}

// Units of all sequences are at most 2^51: bounds that ascend give 2^31 rows, so
// 2^27 + 2^16 tiles, of pairs of up to 2^24 + 4 units.  Bounds that do not would give each
// sequence as many, past 64 bits; one that is below its predecessor counts as
// kDisorder units, and a launch that finds more than kMostUnits does nothing.
// (128 sequences at once, and 256 to a lane of a workgroup, stay below 2^61.)
constexpr int64_t kMostUnits = (int64_t)1 << 52, kDisorder = (int64_t)1 << 53;

// Sequence s if it is one of those with `least` < rows <= `most`; tokens -1 if its bounds are out of order.
__device__ __forceinline__ Sequence sequence(const CacheAttention& a, int s, uint32_t group, uint32_t least, uint32_t most)
{
    Sequence q = {0, 0, 0};
    if (s >= a.c.seqs) return q;
    const int lo = clamp_to(a.c.offsets[s], a.c.tokens), hi = clamp_to(a.c.offsets[s + 1], a.c.tokens);
    if (hi < lo) return {0, -1, 0};
    const uint32_t rows = (uint32_t)(hi - lo) * group;
    if (rows <= least || rows > most) return q;
    return {lo, hi - lo, a.c.pages == 0 ? 0 : seq_length(a.c, s)};
}

// What a workgroup leaves of a cut tile: where it starts, for the joining kernel.
struct Cut {
    int32_t row0, tokens, tile;                  // of the tile; tokens = 0: none begins here
    int32_t parts;                               // in this and the next ranges of the head
};

// The workspace: W cuts, then 2 W parts of R rows: D sums each, then R maxima, R sums of the weights as they are
// multiplied and R of the weights themselves.
template <int D>
__device__ __forceinline__ float* part_of(float* work, unsigned groups, int R, unsigned slot)
{
    return work + (size_t)groups * (sizeof(Cut) / 4) + (size_t)slot * (R * (D + 3));
}

// Rows of tile `tile` that there are, and where row r of q is written.
__device__ __forceinline__ int rows_of(int tokens, int group, int tile, int R)
{
    const int64_t left = (int64_t)tokens * group - (int64_t)tile * R;
    return left < R ? (int)left : R;
}
__device__ __forceinline__ size_t out_row(int row0, uint32_t group, int heads, int head, uint32_t r)
{
    return (size_t)(row0 + r / group) * heads + head * group + r % group;
}

// A row's maximum, the sum of its weights as they are multiplied, rounded, which
// its values are divided by (their errors cancel), and the sum of the weights
// themselves, which the log-sum-exp is formed of.
struct Weights {
    float m, l, exact;
};

// Four values of a row from their sum v and the row's weights.
template <int DT>
__device__ __forceinline__ void write_values(const CacheAttention& a, size_t row, int d, int at, f32x4 v, const Weights& w)
{
    constexpr float kLn2 = 0.693147181f;
    const float f = 1.0f / w.l;
    const f32x4 o = w.l == 0.0f ? f32x4{0, 0, 0, 0} : v * f;
    const size_t i = row * d + at;
    if constexpr (DT == kF32) *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + i) = o;
    else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + i) = u32x2{narrow2<DT>(o[0], o[1]), narrow2<DT>(o[2], o[3])};
    if (a.lse && at == 0) a.lse[row] = w.l == 0.0f ? -__builtin_inff() : (w.m + __builtin_log2f(w.exact)) * kLn2;
}

// The weight that a part of maximum m has under the maximum `most`.
__device__ __forceinline__ float under(float m, float most)
{
    return most == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - most);
}

// How the waves of a workgroup share a tile: its tokens, 32 of a unit each, for
// 16 QT rows; or its rows, 16 QT each, for all tokens.
enum class Share : int { kTokens, kRows };
template <int QT, Share SH> constexpr int kTileRows = 16 * QT * (SH == Share::kRows ? kRowWaves : 1);

// Registers that a lane needs, about: queries, sums, scores, codes, and some.
constexpr int lane_registers(int terms, int nb, int qt)
{
    return qt * (nb * 4 * terms + nb * 8 + 8 + 4 * terms) + (qt == 1 ? 2 : 1) * (nb * 4 + 10) + 60;
}
// Workgroups of a compute unit (waves of a SIMD): by them and by LDS.
constexpr int row_groups(int terms, int nb, int qt)
{
    const int regs = lane_registers(terms, nb, qt), by_regs = regs <= 128 ? 4 : regs <= 168 ? 3 : regs <= 256 ? 2 : 1;
    const int by_lds = 163840 / (kRowWaves * 32 * (nb * 64 + 32) + 4096);
    return by_regs < by_lds ? by_regs : by_lds;
}

// Every wave reads and decodes its tokens by itself: keys pass through LDS as
// codes, from the lanes that asked for them to those that multiply them; values
// pass through it decoded, to be read transposed.
template <int DT, int NB, int QT, Share SH>
__global__ __launch_bounds__(64 * kRowWaves, row_groups(Terms<DT>::v, NB, QT)) void attention_kernel(
    const CacheAttention a, float* work, uint32_t least, uint32_t most_rows)
{
    constexpr int D = 32 * NB, R = kTileRows<QT, SH>, P = Terms<DT>::v, ES = Elem<DT>::size, T = 64 * kRowWaves, ND = D / 16;
    constexpr int kSeqs = 128;                   // sequences looked at at a time
    constexpr int kStride = SH == Share::kTokens ? kUnit : 32;       // tokens from a wave's step to its next
    constexpr int kDepth = SH == Share::kTokens && QT == 1 ? 2 : 1;  // steps asked for ahead
    // kept, addresses would take registers that queries and sums need (16 rows of 256 values: 63 spilled, 20 so), but
    // where there is room they are better kept (prompts, 32 rows of 128 values: 499 us, 457 so)
    constexpr bool kTight = lane_registers(P, NB, QT) > 230 && lane_registers(P, NB, QT) <= 256;
    constexpr float kLog2e = 1.44269504f;
    constexpr bool kExactSum = P < 3;             // three terms are the weight itself
    typedef RowMap<NB> M;
    __shared__ __attribute__((aligned(16))) uint8_t values[kRowWaves][32 * kValueRow<NB>];
    __shared__ int64_t before[kSeqs];            // units before each of them
    __shared__ Sequence seqs[kSeqs];
    __shared__ int64_t sums[kRowWaves];
    __shared__ Weights wave_weights[kRowWaves][16 * QT];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
    const uint32_t group = a.heads / a.c.kv_heads;
    const int kv = a.c.kv_heads;
    // the workgroups of an XCD, every eighth, take neighbouring ranges: they share lines, and tiles of rows what they see
    const unsigned groups = gridDim.x, xcd = blockIdx.x % 8, left = groups % 8;
    const unsigned worker = xcd * (groups / 8) + (xcd < left ? xcd : left) + blockIdx.x / 8;
    const int range = worker / kv, head = worker % kv, most_ranges = groups / kv;

    const auto units_of = [&](const Sequence& q) -> int64_t {
        if (q.tokens < 0) return kDisorder;
        const Tiles t = tiles_of<R>(a, q, group);
        return t.units * t.pairs;
    };
    // sequences s0 .. to LDS, and their units' sum
    const auto look = [&](int s0) -> int64_t {
        __syncthreads();
        int64_t upto = 0, mine = 0;
        if (tid < kSeqs) {
            const Sequence q = sequence(a, s0 + (int)tid, group, least, most_rows);
            seqs[tid] = q;
            upto = mine = units_of(q);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t v = __shfl_up(upto, d, 64);
                if ((int)lane >= d) upto += v;
            }
            if (lane == 63) sums[wave] = upto;
        }
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < kSeqs / 64; ++w) {
            if (w < (int)wave) upto += sums[w];
            total += sums[w];
        }
        if (tid < kSeqs) before[tid] = upto - mine;
        __syncthreads();
        return total;
    };
    int64_t here = look(0), total = here, base = 0;                  // units of the sequences in LDS; all; before those
    if (a.c.seqs > kSeqs) {
        int64_t rest = 0;
        for (int s = kSeqs + (int)tid; s < a.c.seqs; s += T) rest += units_of(sequence(a, s, group, least, most_rows));
        rest = rest < kDisorder ? rest : kDisorder;              // (all lanes' sum fits)
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) rest += __shfl_xor(rest, d, 64);
        if (lane == 0) sums[wave] = rest;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) total += sums[w];
    }
    const int64_t ranges = total > kMostUnits ? 0 : total < most_ranges ? total : most_ranges;
    Cut* const cuts = reinterpret_cast<Cut*>(work);
    if (tid == 0) cuts[worker] = Cut{0, 0, 0, 0};
    if (range >= ranges) return;
    int64_t pos = total * range / ranges;
    const int64_t end = total * (range + 1) / ranges;
    int s0 = 0;
    uint8_t* const mine = values[wave];

    while (pos < end) {
        while (pos >= base + here) {
            base += here;
            s0 += kSeqs;
            if (s0 >= a.c.seqs) return;          // lengths that changed since they were summed up
            here = look(s0);
        }
        int at = 0;                              // the last sequence that begins at or before pos
#pragma unroll
        for (int step = kSeqs / 2; step > 0; step /= 2)
            if (base + before[at + step] <= pos) at += step;
        at = __builtin_amdgcn_readfirstlane(at);
        const Sequence sq = {__builtin_amdgcn_readfirstlane(seqs[at].row0), __builtin_amdgcn_readfirstlane(seqs[at].tokens),
                             __builtin_amdgcn_readfirstlane(seqs[at].length)};
        const Tiles tl = tiles_of<R>(a, sq, group);
        const int64_t rel = pos - base - before[at], item = rel / tl.units, v = rel - item * tl.units;
        int tile = tl.tiles - 1 - (int)item;     // of a pair, the later one first
        Extent ex = extent<R>(a, sq, group, tile);
        int64_t u = v;
        if (u >= ex.units) {
            u -= ex.units;
            tile = tl.tiles - 1 - tile;
            if (tile * 2 + 1 == tl.tiles) ex.units = 0;              // the middle one is alone
            else ex = extent<R>(a, sq, group, tile);
        }
        int64_t n64 = end - pos;
        if (u >= ex.units) {                     // units that stand for nothing
            pos += n64 < tl.units - v ? n64 : tl.units - v;
            continue;
        }
        n64 = n64 < ex.units - u ? n64 : ex.units - u;
        const int u0 = __builtin_amdgcn_readfirstlane((int)u), n = __builtin_amdgcn_readfirstlane((int)n64);
        const int units = __builtin_amdgcn_readfirstlane(ex.units), first = __builtin_amdgcn_readfirstlane(ex.first);
        tile = __builtin_amdgcn_readfirstlane(tile);
        const int rows = rows_of(sq.tokens, group, tile, R);
        // this wave's rows: from r0 on, `own` of them
        const int skip = SH == Share::kRows ? (int)wave * 16 * QT : 0;
        const uint32_t r0 = (uint32_t)tile * R + skip;
        const int own = rows - skip < 16 * QT ? rows - skip : 16 * QT;

        u32x4 fq[QT][NB][P];                     // cut into terms
        int see_lo[QT], see_hi[QT];
        int all_lo = 0, all_hi = 0, any_lo = 0, any_hi = 0;          // what each of the rows sees, and what any does
        if (own > 0) {
            row_sees(a, sq, group, r0, any_lo, all_hi);
            row_sees(a, sq, group, r0 + own - 1, all_lo, any_hi);
        }
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = 16 * t + (int)i;
            const bool in = r < own;
            const uint32_t rr = r0 + (in ? r : 0);
            row_sees(a, sq, group, rr, see_lo[t], see_hi[t]);
            const uint8_t* q = static_cast<const uint8_t*>(a.q) +
                               ((size_t)(sq.row0 + rr / group) * a.q_stride + (size_t)(head * group + rr % group) * D) * ES;
            const uint32_t sign = a.scale < 0 ? 0x80008000u : 0;
#pragma unroll
            for (int s = 0; s < NB; ++s) {
                cut_unit<DT, P>(load_unit<DT>(q + M::unit(s, g) * 8 * ES, in), fq[t][s]);
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int e = 0; e < 4; ++e) fq[t][s][p][e] ^= sign;
            }
        }
        const float c = __builtin_fabsf(a.scale) * kLog2e;

        f32x4 acc[QT][ND];
        f32x4 sum[QT];                           // the weights' sum, four times: a product with ones
        float exact[QT];                         // this lane's weights before they are rounded, if the log-sum-exp is asked for
        float top[QT];                           // the running maximum in binary logarithms
        uint32_t marks[QT];                      // blocks that the row sees not finite
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            top[t] = -__builtin_inff();
            sum[t] = f32x4{0, 0, 0, 0};
            exact[t] = 0.0f;
            marks[t] = 0;
#pragma unroll
            for (int d = 0; d < ND; ++d) acc[t][d] = f32x4{0, 0, 0, 0};
        }

        // this wave's steps of 32 tokens, from key0 on, kStride apart: those that its rows see
        int key0 = first + u0 * kUnit, steps = n;
        if constexpr (SH == Share::kTokens) {
            key0 += (int)wave * 32;
        } else {
            const int key1 = key0 + n * kUnit;   // at most 2^30 + 127
            key0 = any_lo > key0 ? any_lo & ~31 : key0;
            const int last = any_hi < key1 ? any_hi : key1;
            steps = last > key0 ? (last - key0 + 31) / 32 : 0;
        }
        if (sq.length == 0) steps = 0;           // it has no table and may have no page to read
        // where the codes of 32 steps lie, a lane a half step; a step's codes are asked for as soon as those that lie in
        // the same registers, kDepth steps before, are decoded (after the last step, its own again)
        const int32_t* const table = a.c.table + (size_t)(s0 + at) * a.c.max_pages;
        const uint32_t mask16 = (1u << (a.c.shift - 4)) - 1;
        uint32_t where_lo = kNoPage, where_hi = 0;
        struct Ahead {
            Codes<NB> k, v;
            uint32_t ks[2][M::kPieces], vs[kLoads<NB>];
            uint64_t where[2];
        };
        Ahead ahead[kDepth];
        const auto look_up = [&](int step, Ahead& x) {
            if ((step & 31) == 0 && step < steps) {
                const int64_t key = (int64_t)key0 + (int64_t)(step + (int)lane / 2) * kStride + (lane & 1) * 16;
                const int entry = key < sq.length ? table[key >> a.c.shift] : -1;
                const uint64_t w = group_at<NB>(a.c, entry, head, (uint32_t)(key >> 4) & mask16);
                where_lo = (uint32_t)w;
                where_hi = (uint32_t)(w >> 32);
            }
            const int l = (step < steps ? step & 31 : (steps - 1) & 31) * 2;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x.where[h] = (uint64_t)(uint32_t)__builtin_amdgcn_readlane(where_hi, l + h) << 32 | (uint32_t)__builtin_amdgcn_readlane(where_lo, l + h);
        };
        const auto load_keys = [&](Ahead& x) {
            load_codes<NB>(a.c.k, x.where, lane, x.k);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < M::kPieces; ++p) {
                    const uint32_t b = i * NB + M::block(p, g);
                    x.ks[h][p] = kHalves<NB> ? load_scale(tile_at(a.c.k, x.where[h]), b)
                                             : load_scale(tile_at(a.c.k, x.where[0]), block_in(x.where[0]) + h * (16 * NB) + b);
                }
        };
        const auto load_values = [&](Ahead& x) {
            load_codes<NB>(a.c.v, x.where, lane, x.v);
#pragma unroll
            for (int j = 0; j < kLoads<NB>; ++j) {
                const Spot<NB> p = spot_of<NB>(a.c.v, x.where, j, block_of<NB>(j, lane));
                x.vs[j] = load_scale(p.tile, p.block);
            }
        };
        // Tiles of rows wait for the matrix cores, two waves a SIMD: one that feeds them goes before one that forms
        // weights (prompts of 4500 tokens on average, 32 heads of 128: 508 us without, 457 so; chunks 388, 348; but heads
        // of 256, whose one wave a SIMD has none to go before, 1004 and 1040).  Waves that share tokens wait for memory:
        // no difference.
        struct Prefer {
            __device__ __forceinline__ void operator()(int level) const
            {
                if constexpr (SH == Share::kRows) level == 0 ? __builtin_amdgcn_s_setprio(0) : level == 1 ? __builtin_amdgcn_s_setprio(1) : __builtin_amdgcn_s_setprio(2);
            }
        } prefer;
        const auto one_step = [&](int step, Ahead& x) {
            const int key = key0 + step * kStride;
            uint32_t lane = threadIdx.x & 63;
            if constexpr (kTight) asm volatile("" : "+v"(lane));     // addresses are formed from it in every step
            const uint32_t i = lane & 15, g = lane >> 4;
            const bool there[2] = {(x.where[0] & kNoPage) == 0, (x.where[1] & kNoPage) == 0};
            const bool full = there[0] && there[1] && key >= all_lo && key + 32 <= all_hi;
#pragma unroll
            for (int j = 0; j < kLoads<NB>; ++j) {
                const uint32_t b = block_of<NB>(j, lane);
                if (NB % 2 == 0 || j + 1 < kLoads<NB> || lane < 32)
                    *reinterpret_cast<u32x4*>(mine + b / NB * kKeyRow<NB> + b % NB * 16) = x.k.w[j];
            }
            wave_fence();
            uint32_t kw[2][NB];                  // this lane's words of tokens i and 16 + i
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < M::kPieces; ++p) {
                    const uint8_t* const at_k = mine + (16 * h + i) * kKeyRow<NB> + M::block(p, g) * 16 + M::byte(p, g);
                    if (M::words(p) == 4) {
                        const u32x4 v = *reinterpret_cast<const u32x4*>(at_k);
#pragma unroll
                        for (int e = 0; e < 4; ++e) kw[h][(M::first(p) + e) % NB] = v[e];
                    } else if (M::words(p) == 2) {
                        const u32x2 v = *reinterpret_cast<const u32x2*>(at_k);
                        kw[h][M::first(p)] = v.x;
                        kw[h][(M::first(p) + 1) % NB] = v.y;
                    } else {
                        kw[h][M::first(p)] = *reinterpret_cast<const uint32_t*>(at_k);
                    }
                }
            float kscale[2][M::kPieces];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < M::kPieces; ++p) kscale[h][p] = scale_of(x.ks[h][p], i * NB + M::block(p, g));
            look_up(step + kDepth, x);
            load_keys(x);
            prefer(1);
            f32x4 score[QT][2];
#pragma unroll
            for (int t = 0; t < 2 * QT; ++t) score[t / 2][t % 2] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < NB; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 fk = decode8(kw[h][s], kscale[h][M::piece(s)]);
#pragma unroll
                    for (int t = 0; t < QT; ++t)
#pragma unroll
                        for (int p = 0; p < P; ++p) score[t][h] = mfma<false>(fk, fq[t][s][p], score[t][h]);
                }
            wave_fence();
            if (!full) {
#pragma unroll
                for (int j = 0; j < kLoads<NB>; ++j) {
                    // what no row sees counts as zeros; so does a block that is not finite, which would reach the rows
                    // whose weight for it is zero: the rows that see it are marked
                    const uint32_t b = block_of<NB>(j, lane), k = b / NB;
                    const bool in = (k < 16 ? there[0] : there[1]) && key + (int)k >= any_lo && key + (int)k < any_hi;
                    const bool wrong = in && not_finite(x.v.w[j], scale_byte(x.vs[j], b));
                    for (uint64_t left = __builtin_amdgcn_ballot_w64(wrong); left != 0; left &= left - 1) {
                        const int at_b = (int)block_of<NB>(j, __builtin_ctzll(left)), k_b = key + at_b / NB;
#pragma unroll
                        for (int t = 0; t < QT; ++t) marks[t] |= k_b >= see_lo[t] && k_b < see_hi[t] ? 1u << at_b % NB : 0;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) x.v.w[j][e] = in && !wrong ? x.v.w[j][e] : 0;
                    x.vs[j] = in && !wrong ? x.vs[j] : 0x7F7F7F7F;
                }
            }
#pragma unroll
            for (int j = 0; j < kLoads<NB>; ++j) {
                const uint32_t b = block_of<NB>(j, lane);
                const float scale = scale_of(x.vs[j], b);
                uint8_t* const at_v = mine + value_at<NB>(b / NB, b % NB * 4);
                const uint32_t turn = NB == 2 ? b & 1 : b % NB / 2;
                const u32x4 w = turned<NB>(x.v.w[j], turn);
                if (NB % 2 == 0 || j + 1 < kLoads<NB> || lane < 32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) *reinterpret_cast<u32x4*>(at_v + ((e + turn) & 3) * 16) = decode8(w[e], scale);
                }
            }
            wave_fence();
            load_values(x);
            // the first values are read while the weights are formed
            const uint8_t* const column = mine + value_at<NB>(4 * g + i / 4, i % 4 / 2) + i % 2 * 8;
            constexpr int kAhead = 4;
            u32x4 fv[kAhead];
#pragma unroll
            for (int d = 0; d < kAhead; ++d) fv[d] = load_columns(column + 32 * d, 16 * kValueRow<NB>);
            __builtin_amdgcn_sched_barrier(0);
            // weights under the maximum so far, which may lag behind by 2^8; where that is not enough (or there is none
            // yet), or some row does not see all, the maximum is moved, and what is summed under it
            float p[QT][8];
            prefer(0);
            bool late = false;                   // (of any lane: one test of the wave)
#pragma unroll
            for (int t = 0; t < QT; ++t) {
#pragma unroll
                for (int e = 0; e < 8; ++e) p[t][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(score[t][e / 4][e % 4], c, -top[t]));
                late |= !(fmaxf(fmaxf(fmaxf(fmaxf(p[t][0], p[t][1]), p[t][2]), fmaxf(fmaxf(p[t][3], p[t][4]), p[t][5])), fmaxf(p[t][6], p[t][7])) <= 256.0f);
            }
            if (__builtin_expect(__builtin_amdgcn_ballot_w64(late | !full) != 0, 0)) {
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    float most = top[t];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int k = key + 16 * (e / 4) + 4 * (int)g + e % 4;
                        const bool in = there[e / 4] && k >= see_lo[t] && k < see_hi[t];
                        p[t][e] = in ? score[t][e / 4][e % 4] * c : -__builtin_inff();
                        most = fmaxf(most, p[t][e]);
                    }
                    most = max_of_row(most);
                    const float base = most == -__builtin_inff() ? 0.0f : most, f = most == base ? __builtin_amdgcn_exp2f(top[t] - most) : 1.0f;
                    top[t] = most;
#pragma unroll
                    for (int d = 0; d < ND; ++d) acc[t][d] *= f;
                    sum[t] *= f;
                    exact[t] *= f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[t][e] = __builtin_amdgcn_exp2f(p[t][e] - base);
                }
            }
            if (kExactSum && a.lse) {            // (prompts of 4500 tokens on average 468 us, 485 with it)
#pragma unroll
                for (int t = 0; t < QT; ++t)
                    exact[t] += ((p[t][0] + p[t][1]) + (p[t][2] + p[t][3])) + ((p[t][4] + p[t][5]) + (p[t][6] + p[t][7]));
            }
            prefer(2);
            u32x4 fp[QT][P];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                cut_weights<P>(p[t], fp[t]);
#pragma unroll
                for (int y = 0; y < P; ++y) sum[t] = mfma<false>(u32x4{0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80}, fp[t][y], sum[t]);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int p = 0; p < P; ++p) acc[t][d] = mfma<false>(fv[d % kAhead], fp[t][p], acc[t][d]);
                if (d + kAhead < ND) fv[d % kAhead] = load_columns(column + 32 * (d + kAhead), 16 * kValueRow<NB>);
            }
            prefer(0);
            wave_fence();
        };
        if (steps > 0) {
#pragma unroll
            for (int y = 0; y < kDepth; ++y) {
                look_up(y, ahead[y]);
                load_keys(ahead[y]);
                __builtin_amdgcn_sched_barrier(0);               // in the order of the loop, whose waits count them
                load_values(ahead[y]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // (no way leads past one of a turn's steps into the next turn: waits for loads count those of the steps between)
        int step = 0;
        if constexpr (kDepth == 2) {
            for (; step + 1 < steps; step += 2) {
                one_step(step, ahead[0]);
                one_step(step + 1, ahead[1]);
            }
            if (step < steps) one_step(step, ahead[0]);
        } else {
            for (; step < steps; ++step) one_step(step, ahead[0]);
        }

#pragma unroll
        for (int t = 0; t < QT; ++t)
            if (__builtin_expect(__builtin_amdgcn_ballot_w64(marks[t] != 0) != 0, 0)) {
#pragma unroll
                for (int d = 0; d < ND; ++d) acc[t][d] += marks[t] >> (d / 2) & 1 ? __builtin_nanf("") : 0.0f;
            }
        const bool whole = u0 == 0 && n == units;
        float* const part = part_of<D>(work, groups, R, 2 * worker + (u0 == 0 ? 1 : 0));
        // row r of 16, values 4 u .. of it: their sum, the maximum and the weights' sum
        const auto put = [&](int r, int u, f32x4 x, const Weights& w) {
            if (whole) {
                write_values<DT>(a, out_row(sq.row0, group, a.heads, head, r0 + r), D, u * 4, x, w);
            } else {
                *reinterpret_cast<f32x4*>(part + (skip + r) * D + u * 4) = x;
                if (u == 0) { part[R * D + skip + r] = w.m; part[R * D + R + skip + r] = w.l; part[R * D + 2 * R + skip + r] = w.exact; }
            }
        };
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const float all = kExactSum ? sum_of_row(exact[t]) : sum[t][0];
            if (g == 0) wave_weights[wave][16 * t + i] = Weights{top[t], sum[t][0], all};
        }
        float* const o = reinterpret_cast<float*>(mine);             // 16 rows of D sums, 16 bytes apart
        if constexpr (SH == Share::kTokens) {    // the waves' sums meet
            __syncthreads();
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                float most = wave_weights[0][16 * t + i].m;
#pragma unroll
                for (int w = 1; w < kRowWaves; ++w) most = fmaxf(most, wave_weights[w][16 * t + i].m);
                const float f = under(top[t], most);
#pragma unroll
                for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(o + i * (D + 4) + 16 * d + 4 * g) = acc[t][d] * f;
                __syncthreads();
                for (int e = tid; e < 16 * (D / 4); e += T) {
                    const int r = e / (D / 4), u = e % (D / 4);
                    if (16 * t + r >= own) continue;
                    f32x4 x = {0, 0, 0, 0};
                    Weights all = {-__builtin_inff(), 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < kRowWaves; ++w) {
                        x += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(values[w]) + r * (D + 4) + u * 4);
                        all.m = fmaxf(all.m, wave_weights[w][16 * t + r].m);
                    }
#pragma unroll
                    for (int w = 0; w < kRowWaves; ++w) {
                        const Weights& one = wave_weights[w][16 * t + r];
                        const float f = under(one.m, all.m);
                        all.l += one.l * f;
                        all.exact += one.exact * f;
                    }
                    put(16 * t + r, u, x, all);
                }
                __syncthreads();
            }
        } else {
#pragma unroll
            for (int t = 0; t < QT; ++t) {
#pragma unroll
                for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(o + i * (D + 4) + 16 * d + 4 * g) = acc[t][d];
                wave_fence();
                for (int e = lane; e < 16 * (D / 4); e += 64) {
                    const int r = e / (D / 4), u = e % (D / 4);
                    if (16 * t + r < own)
                        put(16 * t + r, u, *reinterpret_cast<const f32x4*>(o + r * (D + 4) + u * 4), wave_weights[wave][16 * t + r]);
                }
                wave_fence();
            }
        }
        if (u0 == 0 && !whole && tid == 0) {
            const int64_t last = pos + units - 1;                    // the tile's last unit
            cuts[worker] = Cut{sq.row0, sq.tokens, tile, (int)(((last + 1) * ranges - 1) / total) - range + 1};
        }
        pos += n;
    }
}

// What a launch of the kernel above leaves: its workspace, workgroups, and rows of a tile.
struct Parts {
    float* work;
    unsigned groups;
    int rows;
};

// Joins the parts of a tile that begins in workgroup blockIdx.x of the first
// launch, or of the second, and is cut, blockIdx.y's rows of it.  D / 4 lanes ask
// for four parts of a row at once; a row of more parts has as many such stripes as
// it needs (few rows of a long sequence lie in many parts), and the rest of the
// workgroup other rows.  One kernel for both launches: 4 us a call less.
template <int DT, int NB>
__global__ __launch_bounds__(256) void attention_join_kernel(const CacheAttention a, const Parts first, const Parts second)
{
    constexpr int D = 32 * NB, L = D / 4, S = 256 / L;
    __shared__ f32x4 sums[S][L];
    __shared__ Weights weights[S];
    const bool later = blockIdx.x >= first.groups;
    const float* const work = later ? second.work : first.work;
    const unsigned groups = later ? second.groups : first.groups, worker = blockIdx.x - (later ? first.groups : 0);
    const int R = later ? second.rows : first.rows;
    const Cut cut = reinterpret_cast<const Cut*>(work)[worker];
    if (cut.tokens == 0) return;
    const int tid = threadIdx.x, at = tid % L, group = a.heads / a.c.kv_heads;
    const int rows = rows_of(cut.tokens, group, cut.tile, R), count = cut.parts, kv = a.c.kv_heads, head = worker % kv;
    const int need = (count + 3) / 4, stripes = need < S ? need : S, at_once = S / stripes;
    const int own = tid / L / stripes, stripe = tid / L % stripes;
    for (int r0 = blockIdx.y * at_once; r0 < rows; r0 += gridDim.y * at_once) {
        const int r = r0 + own;
        const bool in = own < at_once && r < rows;
        Weights w = {-__builtin_inff(), 0.0f, 0.0f};
        f32x4 v = {0, 0, 0, 0};
        for (int x = stripe; in && x < count; x += 4 * stripes) {    // running, as the parts themselves were formed
            Weights pw[4];
            f32x4 pv[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int z = x + y * stripes;
                pw[y] = Weights{-__builtin_inff(), 0.0f, 0.0f};
                pv[y] = f32x4{0, 0, 0, 0};
                if (z < count) {
                    const float* p = part_of<D>(const_cast<float*>(work), groups, R, 2 * (worker + z * kv) + (z == 0 ? 1 : 0));
                    pw[y] = Weights{p[R * D + r], p[R * D + R + r], p[R * D + 2 * R + r]};
                    pv[y] = *reinterpret_cast<const f32x4*>(p + r * D + at * 4);
                }
            }
            const float most = fmaxf(fmaxf(fmaxf(pw[0].m, pw[1].m), fmaxf(pw[2].m, pw[3].m)), w.m), old = under(w.m, most);
            w = Weights{most, w.l * old, w.exact * old};
            v *= old;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float f = under(pw[y].m, most);
                w.l += pw[y].l * f;
                w.exact += pw[y].exact * f;
                v += pv[y] * f;
            }
        }
        if (stripes > 1) {
            const int slot = own * stripes + stripe;
            if (in) {
                sums[slot][at] = v;
                if (at == 0) weights[slot] = w;
            }
            __syncthreads();
            if (in && stripe == 0) {
                float most = w.m;
                for (int x = 1; x < stripes; ++x) most = fmaxf(most, weights[slot + x].m);
                const float own_f = under(w.m, most);
                w = Weights{most, w.l * own_f, w.exact * own_f};
                v *= own_f;
                for (int x = 1; x < stripes; ++x) {
                    const float f = under(weights[slot + x].m, most);
                    v += sums[slot + x][at] * f;
                    w.l += weights[slot + x].l * f;
                    w.exact += weights[slot + x].exact * f;
                }
            }
            __syncthreads();
        }
        if (in && stripe == 0)
            write_values<DT>(a, out_row(cut.row0, group, a.heads, head, (uint32_t)cut.tile * R + r), D, at * 4, v, w);
    }
}

// Workgroups of a launch: whole ranges of all heads, as many as the card's 256
// units hold (a number of its own, as the workspace is sized without a card), or
// one range where there are more heads; and its workspace.
template <int DT, int NB, int QT>
constexpr unsigned attention_groups(size_t kv)
{
    const unsigned fit = 256 * row_groups(Terms<DT>::v, NB, QT), heads = (unsigned)kv;
    return heads < fit ? fit / heads * heads : heads;
}
template <int DT, int NB, int QT, Share SH>
constexpr size_t attention_bytes(size_t kv)
{
    return attention_groups<DT, NB, QT>(kv) * (sizeof(Cut) + 2 * kTileRows<QT, SH> * (32 * NB + 3) * sizeof(float));
}

template <int DT, int NB, int QT, Share SH>
hipError_t attention_launch(const CacheAttention& a, float* work, size_t least, size_t most, Parts& parts, hipStream_t st)
{
    // no more ranges than units that there can be
    const size_t kv = a.c.kv_heads, units = ((size_t)a.c.max_pages << a.c.shift) / kUnit + 1;
    const size_t tiles = ((size_t)a.c.tokens * (a.heads / kv) + kTileRows<QT, SH> - 1) / kTileRows<QT, SH> + a.c.seqs;
    const size_t W = attention_groups<DT, NB, QT>(kv), need = units < W && tiles < W ? units * tiles * kv : W;
    parts = {work, (unsigned)(need < W ? need : W), kTileRows<QT, SH>};
    attention_kernel<DT, NB, QT, SH><<<parts.groups, 64 * kRowWaves, 0, st>>>(a, work, (uint32_t)least, (uint32_t)(most < 0x7FFFFFFF ? most : 0x7FFFFFFF));
    return hipGetLastError();
}

// `rows`: no sequence has more rows of q a head.
template <int DT, int NB>
hipError_t attention_d(const CacheAttention& a, size_t rows, hipStream_t st)
{
    const size_t all = ~(size_t)0;
    Parts first = {}, second = {};
    hipError_t e;
    switch (attention_form(rows, a.c.seqs)) {
    case AttentionForm::kTokens16: e = attention_launch<DT, NB, 1, Share::kTokens>(a, a.work, 0, all, first, st); break;
    case AttentionForm::kTokens32: e = attention_launch<DT, NB, 2, Share::kTokens>(a, a.work, 0, all, first, st); break;
    case AttentionForm::kRows: e = attention_launch<DT, NB, 2, Share::kRows>(a, a.work, 0, all, first, st); break;
    default:
        e = attention_launch<DT, NB, 2, Share::kRows>(a, a.work, kFewRows, all, first, st);
        if (e != hipSuccess) return e;
        float* const behind = a.work + attention_bytes<DT, NB, 2, Share::kRows>(a.c.kv_heads) / 4;
        e = attention_launch<DT, NB, 2, Share::kTokens>(a, behind, 0, kFewRows, second, st);
    }
    if (e != hipSuccess) return e;
    attention_join_kernel<DT, NB><<<dim3(first.groups + second.groups, 4), 256, 0, st>>>(a, first, second);
    return hipGetLastError();
}

template <int DT, int NB>
size_t attention_work_d(size_t rows, size_t kv)
{
    const size_t few = attention_bytes<DT, NB, 1, Share::kTokens>(kv), some = attention_bytes<DT, NB, 2, Share::kTokens>(kv);
    if (rows <= 16) return few;
    // a hint may ask for the kernel of 16 rows all the same
    if (rows <= kFewRows) return some > few ? some : few;
    const size_t many = attention_bytes<DT, NB, 2, Share::kRows>(kv) + some;
    return many > few ? many : few;
}

template <int DT>
hipError_t attention_t(int d, const CacheAttention& a, size_t rows, hipStream_t st)
{
    switch (d) {
    case 64: return attention_d<DT, 2>(a, rows, st);
    case 96: return attention_d<DT, 3>(a, rows, st);
    case 128: return attention_d<DT, 4>(a, rows, st);
    case 192: return attention_d<DT, 6>(a, rows, st);
    default: return attention_d<DT, 8>(a, rows, st);
    }
}

template <int DT>
size_t attention_work_t(int d, size_t rows, size_t kv)
{
    switch (d) {
    case 64: return attention_work_d<DT, 2>(rows, kv);
    case 96: return attention_work_d<DT, 3>(rows, kv);
    case 128: return attention_work_d<DT, 4>(rows, kv);
    case 192: return attention_work_d<DT, 6>(rows, kv);
    case 256: return attention_work_d<DT, 8>(rows, kv);
    default: return 0;
    }
}

}  // namespace rc
