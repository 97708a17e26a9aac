// rc_op_cache.hpp -- where a row stands in a paged cache, and where the cache
// holds a token, shared by the kernels that write and read it.
#pragma once

#include "rc_op.hpp"
#include "rc_op_launch.hpp"

namespace rc {

constexpr uint32_t kMxTile = 1088;               // an MXFP4 tile: 1024 bytes of codes, 64 scales

__device__ __forceinline__ int clamp_to(int v, int most) { return v < 0 ? 0 : v > most ? most : v; }

// Tokens of a sequence in the cache.
__device__ __forceinline__ int seq_length(const Cache& c, int s) { return clamp_to(c.lengths[s], c.max_pages << c.shift); }

// Byte of block b's codes (its eight-value units are 4 bytes each) and of its
// scale in a head's stream of one page.
__device__ __forceinline__ uint32_t codes_at(uint32_t b) { return b / 64 * kMxTile + b % 64 * 16; }
__device__ __forceinline__ uint32_t scale_at(uint32_t b) { return b / 64 * kMxTile + 1024 + b % 64; }

// Byte of a head's stream in a page (pages x kv_heads streams).
__device__ __forceinline__ size_t stream_at(const Cache& c, int page, int head)
{
    return ((size_t)page * c.kv_heads + head) * c.head_bytes;
}

// The sequence of row i and the row's position, -1 if it belongs to none: the
// first bound above i is looked for by all lanes at once, 64 bounds a round.
// Wave-uniform.
struct RowPlace { int seq, pos; };
__device__ __forceinline__ RowPlace row_place(const Cache& c, int i)
{
    const int lane = threadIdx.x & 63;
    int lo = 0, n = c.seqs;
    for (;;) {
        const int step = (n + 63) / 64, at = lo + (lane + 1) * step - 1, last = lo + n - 1;
        const bool past = lane * step < n && clamp_to(c.offsets[(at < last ? at : last) + 1], c.tokens) > i;
        const uint64_t b = __builtin_amdgcn_ballot_w64(past);
        if (b == 0) return {-1, -1};
        const int l = __builtin_ctzll(b);
        lo += l * step;
        n = step < n - l * step ? step : n - l * step;
        if (step == 1) break;
    }
    const int s = __builtin_amdgcn_readfirstlane(lo);
    const int end = clamp_to(c.offsets[s + 1], c.tokens);
    if (clamp_to(c.offsets[s], c.tokens) > i) return {-1, -1};
    return {s, seq_length(c, s) - end + i};
}

// The page of position pos of sequence s, -1 if there is none.
__device__ __forceinline__ int page_of(const Cache& c, int s, int pos)
{
    if (pos < 0) return -1;
    const int p = c.table[(size_t)s * c.max_pages + (pos >> c.shift)];
    return p >= 0 && p < c.pages ? p : -1;
}

}  // namespace rc
