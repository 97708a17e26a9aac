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
// weights exp(s_j - m): one term rounds them to 2^-9 of themselves, which is
// less than what rounding the result to bfloat16 costs, as its errors average out.
#pragma once

#include "rc_op_cache.hpp"
#include "rc_op_matrix.hpp"

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

// A lane's part of sixteen tokens' codes.
template <int NB>
struct Codes {
    uint32_t w[NB], s[RowMap<NB>::kPieces];
};

// Asks for tokens 16 k .. of a page's stream; lane (i, g) has token 16 k + i.
template <int NB>
__device__ __forceinline__ void load_codes(const uint8_t* stream, uint32_t k, uint32_t i, uint32_t g, Codes<NB>& c)
{
    typedef RowMap<NB> M;
    const uint32_t b0 = 16 * NB * k, rem = NB % 4 == 0 ? 0 : b0 % 64;
    const uint8_t* tile = stream + b0 / 64 * kMxTile;
#pragma unroll
    for (int p = 0; p < M::kPieces; ++p) {
        const uint32_t b = rem + i * NB + M::block(p, g);
        const uint8_t* at = tile + codes_at(b) + M::byte(p, g);
        if (M::words(p) == 4) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(at);
#pragma unroll
            for (int e = 0; e < 4; ++e) c.w[(M::first(p) + e) % NB] = v[e];
        } else if (M::words(p) == 2) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(at);
            c.w[M::first(p)] = v.x;
            c.w[(M::first(p) + 1) % NB] = v.y;
        } else {
            c.w[M::first(p)] = *reinterpret_cast<const uint32_t*>(at);
        }
        c.s[p] = tile[scale_at(b)];
    }
}

// ---- values in LDS: rows of D bfloat16 values, one a token, in 16-byte units
// that are swizzled by the token so that the lanes of a store (eight tokens, one
// unit) and of a transposing load (eight tokens, two units) fall on all banks.
template <int NB>
__device__ __forceinline__ uint32_t swizzle(uint32_t token)
{
    return NB % 4 == 0 ? (token & 7) * 2 : NB % 2 == 0 ? (token >> 1 & 3) * 2 : (token >> 2 & 1) * 2;
}
template <int NB>
__device__ __forceinline__ uint32_t value_at(uint32_t token, uint32_t unit)
{
    return token * (NB * 64) + ((unit ^ swizzle<NB>(token)) << 4);
}

// Largest over the four lanes that share a row, in each of them.
__device__ __forceinline__ float max_of_row(float v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_of_row(float v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Weights of 2 x 4 tokens as P bfloat16 terms that add up to them (to 2^-9,
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
// A sequence's items are its row tiles times the cache's heads, an item's units
// its tokens 128 at a time; all units of all sequences stand in one row, and
// workgroup w of W takes the w-th part of them, so that sequences of all lengths
// load the card alike.  An item that is cut is joined by a second kernel: a
// workgroup leaves at most two parts, of the item that it takes over (slot 2 w)
// and of the one that it leaves (slot 2 w + 1).
struct Sequence {
    int row0, tokens, length, first;             // rows of q; tokens in the cache, and the first that any row sees
    int units, tiles;                            // of an item; of rows
};

template <int R>
__device__ __forceinline__ Sequence sequence(const CacheAttention& a, int s)
{
    Sequence q = {0, 0, 0, 0, 0, 0};
    if (s >= a.c.seqs) return q;
    const int lo = clamp_to(a.c.offsets[s], a.c.tokens), hi = clamp_to(a.c.offsets[s + 1], a.c.tokens);
    if (hi <= lo) return q;
    q.row0 = lo;
    q.tokens = hi - lo;
    q.length = a.c.pages == 0 ? 0 : seq_length(a.c, s);
    const int64_t see = (int64_t)q.length - q.tokens - a.window + 1;
    q.first = a.window != 0 && see > 0 ? (int)(see & ~(int64_t)31) : 0;
    q.units = (q.length - q.first + kUnit - 1) / kUnit;
    if (q.units < 1) q.units = 1;                // its rows are written all the same
    q.tiles = (int)(((int64_t)q.tokens * (a.heads / a.c.kv_heads) + R - 1) / R);
    return q;
}

// What a workgroup leaves of a cut item: where it starts, for the joining kernel.
struct Cut {
    int32_t row0, tokens, tile, head;            // as in the item; tokens = 0: nothing begins here
    int32_t last, pad[3];                        // the last workgroup that has a part of it
};

// The workspace: W cuts, then 2 W parts of R rows: D sums each, then R maxima, R sums of weights.
template <int D, int R>
__device__ __forceinline__ float* part_of(float* work, unsigned groups, unsigned slot)
{
    return work + (size_t)groups * (sizeof(Cut) / 4) + (size_t)slot * (R * (D + 2));
}

// Rows r of tile `tile` that there are, and where row r is written.
__device__ __forceinline__ int rows_of(int tokens, int group, int tile, int R)
{
    const int64_t left = (int64_t)tokens * group - (int64_t)tile * R;
    return left < R ? (int)left : R;
}
__device__ __forceinline__ size_t out_row(int row0, uint32_t group, int heads, int head, uint32_t r)
{
    return (size_t)(row0 + r / group) * heads + head * group + r % group;
}

// Four values of a row from their sum v, the sum l of the weights and the maximum m.
template <int DT>
__device__ __forceinline__ void write_values(const CacheAttention& a, size_t row, int d, int at, f32x4 v, float m, float l)
{
    constexpr float kLn2 = 0.693147181f;
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    const f32x4 o = l == 0.0f ? f32x4{0, 0, 0, 0} : v * f;
    const size_t i = row * d + at;
    if constexpr (DT == kF32) *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + i) = o;
    else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + i) = u32x2{narrow2<DT>(o[0], o[1]), narrow2<DT>(o[2], o[3])};
    if (a.lse && at == 0) a.lse[row] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
}

// Workgroups of a compute unit (waves of a SIMD), by the registers that a lane
// needs: queries, sums, two steps' codes, and some.
constexpr int row_groups(int terms, int nb, int qt)
{
    const int regs = qt * (nb * 4 * terms + nb * 8) + 2 * (nb * 4 + 10) + 44;
    return regs <= 128 ? 4 : regs <= 168 ? 3 : regs <= 256 ? 2 : 1;
}

// Few rows an item: every wave takes 32 tokens of a unit, reads and decodes them
// by itself and keeps 16 QT rows of q; the waves' sums meet at the item's end.
// Keys go from memory to the registers that the matrix instructions read;
// values pass through LDS, decoded, to be read transposed.
template <int DT, int NB, int QT>
__global__ __launch_bounds__(64 * kRowWaves, row_groups(Terms<DT>::v, NB, QT)) void attention_rows_kernel(const CacheAttention a)
{
    constexpr int D = 32 * NB, R = 16 * QT, P = Terms<DT>::v, ES = Elem<DT>::size, T = 64 * kRowWaves, ND = D / 16;
    constexpr float kLog2e = 1.44269504f;
    typedef RowMap<NB> M;
    __shared__ __attribute__((aligned(16))) uint8_t values[kRowWaves][32 * D * 2];
    __shared__ int64_t before[T];                // units before each of 256 sequences
    __shared__ Sequence seqs[T];
    __shared__ int64_t sums[kRowWaves];
    __shared__ float wave_max[kRowWaves][R], wave_sum[kRowWaves][R];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
    const int group = a.heads / a.c.kv_heads, kv = a.c.kv_heads;
    const unsigned groups = gridDim.x;

    // sequences s0 .. s0 + 255 to LDS, and their units' sum
    auto look = [&](int s0) -> int64_t {
        __syncthreads();
        const Sequence q = sequence<R>(a, s0 + (int)tid);
        seqs[tid] = q;
        int64_t upto = (int64_t)q.units * q.tiles * kv;
        const int64_t mine = upto;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t v = __shfl_up(upto, d, 64);
            if ((int)lane >= d) upto += v;
        }
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) {
            if (w < (int)wave) upto += sums[w];
            total += sums[w];
        }
        before[tid] = upto - mine;
        __syncthreads();
        return total;
    };
    int64_t total = 0, base = 0, here = 0;       // units; before the sequences in LDS; of them
    for (int s0 = 0; s0 < a.c.seqs; s0 += T) { here = look(s0); total += here; }
    const int64_t workers = total < groups ? total : groups;
    Cut* const cuts = reinterpret_cast<Cut*>(a.work);
    if (tid == 0) cuts[blockIdx.x] = Cut{0, 0, 0, 0, 0, {0, 0, 0}};
    if (blockIdx.x >= workers) return;
    int64_t pos = total * blockIdx.x / workers;
    const int64_t end = total * (blockIdx.x + 1) / workers;
    int s0 = 0;
    if (a.c.seqs > T) here = look(0);

    uint8_t* const mine = values[wave];
    while (pos < end) {
        while (pos >= base + here) { base += here; s0 += T; here = look(s0); }
        // the last sequence that begins at or before pos and has units
        int lo = 0;
#pragma unroll
        for (int step = T / 2; step > 0; step /= 2)
            if (base + before[lo + step] <= pos) lo += step;
        lo = __builtin_amdgcn_readfirstlane(lo);
        const Sequence sq = seqs[lo];
        const int row0 = __builtin_amdgcn_readfirstlane(sq.row0), tokens = __builtin_amdgcn_readfirstlane(sq.tokens);
        const int length = __builtin_amdgcn_readfirstlane(sq.length), first = __builtin_amdgcn_readfirstlane(sq.first);
        const int units = __builtin_amdgcn_readfirstlane(sq.units);
        const int64_t rel = pos - base - before[lo], item = rel / units;
        const int u0 = __builtin_amdgcn_readfirstlane((int)(rel - item * units));
        const int head = __builtin_amdgcn_readfirstlane((int)(item % kv)), tile = __builtin_amdgcn_readfirstlane((int)(item / kv));
        const int n = __builtin_amdgcn_readfirstlane((int)(end - pos < units - u0 ? end - pos : units - u0));
        const int rows = rows_of(tokens, group, tile, R);
        const uint32_t r0 = (uint32_t)tile * R;   // tokens * heads is below 2^31

        // this lane's rows: their positions' bounds, their values cut into terms
        u32x4 fq[QT][NB][P];
        int see_lo[QT], see_hi[QT];
        const auto bounds = [&](uint32_t r, int& lo_, int& hi_) {
            const int64_t p = (int64_t)length - tokens + r / (uint32_t)group;
            hi_ = a.causal ? (p < length ? (int)(p + 1 < 0 ? 0 : p + 1) : length) : length;
            lo_ = a.window && p - a.window + 1 > 0 ? (int)(p - a.window + 1) : 0;
        };
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = 16 * t + i;
            const bool in = r < rows;
            const uint32_t rr = r0 + (in ? r : rows - 1);
            bounds(rr, see_lo[t], see_hi[t]);
            const uint8_t* q = static_cast<const uint8_t*>(a.q) +
                               ((size_t)(row0 + rr / (uint32_t)group) * a.q_stride + (size_t)(head * group + rr % (uint32_t)group) * D) * ES;
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
        int all_lo, all_hi, any_lo, any_hi;       // what every row of the tile sees, and what any does
        bounds(r0, any_lo, all_hi);
        bounds(r0 + rows - 1, all_lo, any_hi);
        const float c = __builtin_fabsf(a.scale) * kLog2e;

        f32x4 acc[QT][ND];
        float top[QT], sum[QT];                   // the running maximum in binary logarithms; this lane's part of the sum
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            top[t] = -__builtin_inff();
            sum[t] = 0.0f;
#pragma unroll
            for (int d = 0; d < ND; ++d) acc[t][d] = f32x4{0, 0, 0, 0};
        }

        // the table's entries of this wave's next 32 steps, a lane a half step
        const int seq = s0 + lo;
        const int32_t* table = a.c.table + (size_t)seq * a.c.max_pages;
        const int key0 = first + (u0 * kRowWaves + (int)wave) * 32;
        int pages = -1;
        auto look_up = [&](int step) {
            const int64_t key = (int64_t)key0 + (int64_t)(step + (int)lane / 2) * kUnit + (lane & 1) * 16;
            pages = key < length ? table[key >> a.c.shift] : -1;
            if (pages >= a.c.pages) pages = -1;
        };
        struct Step { Codes<NB> k[2], v[2]; int page[2]; };
        const int mask16 = (1 << (a.c.shift - 4)) - 1;
        auto load = [&](int step, Step& x) {
            if ((step & 31) == 0) look_up(step);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x.page[h] = __builtin_amdgcn_readlane(pages, (step & 31) * 2 + h);
                const int key = key0 + step * kUnit + 16 * h;
                const size_t at = stream_at(a.c, x.page[h] < 0 ? 0 : x.page[h], head);
                const uint32_t k16 = (uint32_t)(key >> 4) & mask16;
                load_codes<NB>(a.c.k + at, k16, i, g, x.k[h]);
                load_codes<NB>(a.c.v + at, k16, i, g, x.v[h]);
            }
        };
        auto compute = [&](int step, Step& x) {
            const int key = key0 + step * kUnit;
            const bool full = x.page[0] >= 0 && x.page[1] >= 0 && key >= all_lo && key + 32 <= all_hi;
            bool odd = false;                     // values that may not be finite where some row does not see them
            if (!full) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int mine_key = key + 16 * h + (int)i;
                    const bool in = x.page[h] >= 0 && mine_key >= any_lo && mine_key < any_hi;
#pragma unroll
                    for (int s = 0; s < NB; ++s) x.v[h].w[s] = in ? x.v[h].w[s] : 0;
#pragma unroll
                    for (int p = 0; p < M::kPieces; ++p) {
                        x.v[h].s[p] = in ? x.v[h].s[p] : 127;
                        odd |= x.v[h].s[p] >= 253;
                    }
                }
                odd = __builtin_amdgcn_ballot_w64(odd) != 0;
            }
            f32x4 score[QT][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int t = 0; t < QT; ++t) score[t][h] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < NB; ++s) {
                    const u32x4 fk = decode8(x.k[h].w[s], __uint_as_float(x.k[h].s[M::piece(s)] << 23));
#pragma unroll
                    for (int t = 0; t < QT; ++t)
#pragma unroll
                        for (int p = 0; p < P; ++p) score[t][h] = mfma<false>(fk, fq[t][s][p], score[t][h]);
                }
#pragma unroll
                for (int s = 0; s < NB; ++s)
                    *reinterpret_cast<u32x4*>(mine + value_at<NB>(16 * h + i, M::unit(s, g))) =
                        decode8(x.v[h].w[s], __uint_as_float(x.v[h].s[M::piece(s)] << 23));
            }
            wave_fence();
            u32x4 fp[QT][P];
            uint32_t seen[QT];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                float p[8];
                float cc = c;
                seen[t] = 0xFF;
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = score[t][e / 4][e % 4];
                if (!full) {
                    seen[t] = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int k = key + 16 * (e / 4) + 4 * (int)g + e % 4;
                        const bool in = x.page[e / 4] >= 0 && k >= see_lo[t] && k < see_hi[t];
                        seen[t] |= in ? 1u << e : 0;
                        p[e] = in ? p[e] * c : -__builtin_inff();
                    }
                    cc = 1.0f;
                }
                float most = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7]))) * cc;
                // the maximum may lag by 2^8: it is moved, and what is summed with it, only when it has to be
                if (__builtin_amdgcn_ballot_w64(most > top[t] + 8.0f) != 0) {
                    most = fmaxf(max_of_row(most), top[t]);
                    const float old = most == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top[t] - most);
                    top[t] = most;
                    sum[t] *= old;
#pragma unroll
                    for (int d = 0; d < ND; ++d) acc[t][d] *= old;
                }
                const float m = top[t] == -__builtin_inff() ? 0.0f : top[t];
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[e], cc, -m));
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[t] += p[e];
                cut_weights<P>(p, fp[t]);
            }
            auto products = [&](int d, u32x4 fv) {
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int p = 0; p < P; ++p) acc[t][d] = mfma<false>(fv, fp[t][p], acc[t][d]);
            };
            if (!odd) {
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    products(d, load_columns(mine + value_at<NB>(4 * g + i / 4, 2 * d + i % 4 / 2) + i % 2 * 8, 16 * D * 2));
            } else {                              // token by token, for the rows that see it alone
                for (int k = 0; k < 32; ++k) {
                    const bool held = (int)g == k % 16 / 4;
                    const int word = k / 16 * 2 + k % 4 / 2;
                    const uint32_t keep = k % 2 ? 0xFFFF0000u : 0x0000FFFFu;
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        u32x4 fv = load_columns(mine + value_at<NB>(4 * g + i / 4, 2 * d + i % 4 / 2) + i % 2 * 8, 16 * D * 2);
#pragma unroll
                        for (int e = 0; e < 4; ++e) fv[e] = held && e == word ? fv[e] & keep : 0;
#pragma unroll
                        for (int t = 0; t < QT; ++t) {
                            f32x4 one = {0, 0, 0, 0};
#pragma unroll
                            for (int p = 0; p < P; ++p) one = mfma<false>(fv, fp[t][p], one);
                            // the row's lane that has the token's score says whether it is seen
                            const uint32_t bits = (uint32_t)__shfl((int)seen[t], (int)(k % 16 / 4 * 16 + i), 64);
                            const bool in = bits >> (k / 16 * 4 + k % 4) & 1;
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[t][d][e] = in ? acc[t][d][e] + one[e] : acc[t][d][e];
                        }
                    }
                }
            }
            wave_fence();
        };
        Step x, y;
        const int steps = length > 0 ? n : 0;    // an empty sequence has no table and may have no page to read
        if (steps > 0) load(0, x);
        for (int step = 0; step < steps; step += 2) {
            if (step + 1 < steps) load(step + 1, y);
            compute(step, x);
            if (step + 1 >= steps) break;
            if (step + 2 < steps) load(step + 2, x);
            compute(step + 1, y);
        }

        // the waves' sums meet
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            sum[t] = sum_of_row(sum[t]);
            if (g == 0) { wave_max[wave][16 * t + i] = top[t]; wave_sum[wave][16 * t + i] = sum[t]; }
        }
        __syncthreads();
        const bool whole = u0 == 0 && n == units;
        float* const part = part_of<D, R>(a.work, groups, 2 * blockIdx.x + (u0 == 0 ? 1 : 0));
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            float most = wave_max[0][16 * t + i];
#pragma unroll
            for (int w = 1; w < kRowWaves; ++w) most = fmaxf(most, wave_max[w][16 * t + i]);
            const float f = most == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(top[t] - most);
            float* const o = reinterpret_cast<float*>(mine);        // 16 rows of D sums
#pragma unroll
            for (int d = 0; d < ND; ++d)
                *reinterpret_cast<f32x4*>(o + i * D + (((4 * d + g) ^ (i & 7)) << 2)) = acc[t][d] * f;
            __syncthreads();
            for (int e = tid; e < 16 * (D / 4); e += T) {
                const int r = e / (D / 4), u = e % (D / 4);
                if (16 * t + r >= rows) continue;
                f32x4 v = {0, 0, 0, 0};
                float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
                for (int w = 0; w < kRowWaves; ++w) {
                    v += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(values[w]) + r * D + ((u ^ (r & 7)) << 2));
                    m = fmaxf(m, wave_max[w][16 * t + r]);
                }
#pragma unroll
                for (int w = 0; w < kRowWaves; ++w)
                    l += wave_sum[w][16 * t + r] * (m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(wave_max[w][16 * t + r] - m));
                if (whole) {
                    const size_t at = out_row(row0, group, a.heads, head, r0 + 16 * t + r);
                    write_values<DT>(a, at, D, u * 4, v, m, l);
                } else {
                    *reinterpret_cast<f32x4*>(part + (16 * t + r) * D + u * 4) = v;
                    if (u == 0) { part[R * D + 16 * t + r] = m; part[R * D + R + 16 * t + r] = l; }
                }
            }
            __syncthreads();
        }
        if (u0 == 0 && !whole && tid == 0) {
            const int64_t last = pos + units - 1;                   // the item's last unit
            cuts[blockIdx.x] = Cut{row0, tokens, tile, head, (int)(((last + 1) * workers - 1) / total), {0, 0, 0}};
        }
        pos += n;
    }
}

// Joins the parts of an item that begins in workgroup blockIdx.x and is cut: a wave a row.
template <int DT, int NB, int QT>
__global__ __launch_bounds__(64 * kRowWaves) void attention_join_kernel(const CacheAttention a, unsigned groups)
{
    constexpr int D = 32 * NB, R = 16 * QT;
    const Cut cut = reinterpret_cast<const Cut*>(a.work)[blockIdx.x];
    if (cut.tokens == 0) return;
    const int lane = threadIdx.x & 63, group = a.heads / a.c.kv_heads, rows = rows_of(cut.tokens, group, cut.tile, R);
    const int count = cut.last - (int)blockIdx.x + 1;
    const auto part = [&](int x) { return part_of<D, R>(a.work, groups, 2 * (blockIdx.x + x) + (x == 0 ? 1 : 0)); };
    for (int r = threadIdx.x >> 6; r < rows; r += kRowWaves) {
        float m = -__builtin_inff();
        for (int x = lane; x < count; x += 64) m = fmaxf(m, part(x)[R * D + r]);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
        float l = 0.0f;
        f32x4 v = {0, 0, 0, 0};
        for (int x = 0; x < count; ++x) {
            const float* p = part(x);
            const float f = m == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(p[R * D + r] - m);
            l += p[R * D + R + r] * f;
            if (lane < D / 4) v += *reinterpret_cast<const f32x4*>(p + r * D + lane * 4) * f;
        }
        if (lane < D / 4) write_values<DT>(a, out_row(cut.row0, group, a.heads, cut.head, (uint32_t)cut.tile * R + r), D, lane * 4, v, m, l);
    }
}

template <int DT, int NB, int QT>
hipError_t attention_rows(const CacheAttention& a, hipStream_t st)
{
    constexpr unsigned W = 256 * row_groups(Terms<DT>::v, NB, QT);
    attention_rows_kernel<DT, NB, QT><<<W, 64 * kRowWaves, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    attention_join_kernel<DT, NB, QT><<<W, 64 * kRowWaves, 0, st>>>(a, W);
    return hipGetLastError();
}

template <int DT, int NB>
hipError_t attention_d(const CacheAttention& a, size_t most_rows, hipStream_t st)
{
    return most_rows <= 16 ? attention_rows<DT, NB, 1>(a, st) : attention_rows<DT, NB, 2>(a, st);
}

template <int DT>
hipError_t attention_t(int d, const CacheAttention& a, size_t most_rows, hipStream_t st)
{
    switch (d) {
    case 64: return attention_d<DT, 2>(a, most_rows, st);
    case 96: return attention_d<DT, 3>(a, most_rows, st);
    case 128: return attention_d<DT, 4>(a, most_rows, st);
    case 192: return attention_d<DT, 6>(a, most_rows, st);
    default: return attention_d<DT, 8>(a, most_rows, st);
    }
}

}  // namespace rc
