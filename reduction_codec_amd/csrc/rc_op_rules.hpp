// rc_op_rules.hpp -- which kernel a product grouped by expert takes: rules on
// sizes and types alone, without HIP, so that a host program can ask them too.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace rc {

struct GroupedSizes { size_t rows, experts; int64_t n, k; };

inline size_t mean_rows(const GroupedSizes& s) { return (s.rows + s.experts - 1) / s.experts; }

// Workgroups, about, for tiles of so many rows by so many of the result's `width` columns.
inline size_t tile_groups(const GroupedSizes& s, int64_t width, size_t rows, size_t columns)
{
    return std::min(s.rows, s.rows / rows + s.experts) * (((size_t)width + columns - 1) / columns);
}

// Forward.  The mean rows of an expert choose how many rows a workgroup takes
// (the weights are read and decoded once per 16 MF rows, but rows that are not
// there cost as much as others), the number of workgroups how they are cut.
// bf16, 32 experts of 2048 x 4096, in us with 16, 32, 64, 128 rows: mean 6: 40,
// 39, 45, -; mean 16: 51, 51, 55, -; mean 64: 114, 87, 83, 105; mean 128: -, -,
// 124, 130; mean 256: -, -, 208, 194.  128 x 256 tiles pay once there are
// several rounds of them: 16384 rows of 8192 x 4096 1110 us -> 1073, but 8192
// rows of 2048 x 4096 177 -> 192.  With few workgroups more and smaller ones:
// 600 rows of 1000 x 2080 15 us with 32 rows, 22 with 64; 2331 and 6000 rows 27
// and 45 with 64 x 256, 30 and 48 with 128 x 128, 33 and 59 with 64 x 128.
// There two groups of waves with every second span each did not help (2331 rows
// 27 us either way in bf16, 28 -> 33 in fp16), nor did waves split over rows
// too, in any tile (16384 rows 1104 -> 1422).
// Three terms take LDS and registers, so fp32 stays with 32 rows: mean 64 with
// 32 x 128, 32 x 256, 64 x 256: 160, 145, 174.  Fewer still leave the card
// idle, and the contraction is cut instead: two rows of 4096 x 4096 take 8 us
// so, 14 us otherwise; 248 workgroups 9.4 and 8.2 us.
//
// The forms: rows by columns of a workgroup, and the 32-wide blocks of a span.
enum class Forward : int {
    kThin16x32, k16x128, k32x128Span16, k32x128Span8, k64x128, k64x256, k128x128, k128x256, k32x128F32, k32x256F32
};

inline Forward forward_form(bool f32, const GroupedSizes& s)
{
    const size_t mean = mean_rows(s);
    const auto groups = [&](size_t rows, size_t columns) { return tile_groups(s, s.n, rows, columns); };
    if (groups(16, 128) < 192) return Forward::kThin16x32;
    if (mean <= 8) return Forward::k16x128;
    if (f32) return mean <= 40 || groups(64, 256) < 128 ? Forward::k32x128F32 : Forward::k32x256F32;
    if (mean <= 40) return Forward::k32x128Span16;
    if (groups(64, 128) < 256) return Forward::k32x128Span8;
    if (mean <= 160) return Forward::k64x128;
    if (groups(64, 256) < 768) return Forward::k64x256;
    if (groups(128, 256) < 1024) return Forward::k128x128;
    return Forward::k128x256;
}

// Gradients.  dx: 64 x 128 tiles until there are enough of 128 x 256; 16 experts
// of 2048 x 4096 in bf16, in us: mean 8: 32, 40; mean 64: 45, 53; mean 72: 57,
// 53; mean 128: 75, 62; mean 256: 125, 99; mean 512: 225, 166; 4282 rows on two
// experts of 6856 x 256 74, 126; 4096 rows on 8 of 1024 x 1024 (160 large tiles)
// 23, 25.  Very few: four
// groups of waves share the contraction, 37 rows of 3624 x 128 37 -> 19 us, 32
// rows over 4 experts of 1024 x 1024 12.7 -> 8.2, but 138 tiles 74 -> 80.  fp16
// with 64 x 128 and 128 x 256: mean 64 68, 100; mean 128 120, 123; mean 256 196,
// 187; mean 512 348, 312.
// dW, 256 x 256 and 128 x 128: 64 large tiles 18, 10; 128: 34, 22; 320: 30, 25;
// 640: 51, 57; 2048: 222, 267.
enum class Dx : int { k64x64Shared, k64x128, k128x256 };

inline Dx dx_form(bool bf16, const GroupedSizes& s)
{
    if (tile_groups(s, s.k, 64, 128) < 100) return Dx::k64x64Shared;
    if (mean_rows(s) <= (bf16 ? 64 : 128) || tile_groups(s, s.k, 128, 256) < 256) return Dx::k64x128;
    return Dx::k128x256;
}

enum class Dw : int { k128x128F32, k128x128, k256x256 };

inline Dw dw_form(bool f32, const GroupedSizes& s)
{
    if (f32) return Dw::k128x128F32;
    return (size_t)((s.n + 255) / 256) * (size_t)((s.k + 255) / 256) * s.experts < 512 ? Dw::k128x128 : Dw::k256x256;
}

}  // namespace rc
