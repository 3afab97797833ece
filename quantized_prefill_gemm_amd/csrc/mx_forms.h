// Which form of the MXFP4 product a shape takes, and its launch: host code without HIP, so that it
// can be looked at without a GPU. The kernels are in mmq_mxfp4.hip.
#pragma once

#include <stdint.h>

namespace qpg {

enum class Form { S16x16, S16x32, S32x16, S32x32, T64, T64x128, T128, T256 };

// Tile (tokens x weight rows), threads of a workgroup, and of the tiled forms the workgroups of a
// grid for each of the 256 CUs (0: a streaming form, a workgroup to a tile).
struct FormShape {
    int bm, bn, threads, per_cu;
};

constexpr FormShape form_shape(Form form)
{
    switch (form) {
    case Form::S16x16: return {16, 16, 512, 0};
    case Form::S16x32: return {16, 32, 256, 0};
    case Form::S32x16: return {32, 16, 512, 0};
    case Form::S32x32: return {32, 32, 512, 0};
    case Form::T64: return {64, 64, 256, 3};
    case Form::T64x128: return {64, 128, 256, 2};
    case Form::T128: return {128, 128, 256, 2};
    default: return {256, 256, 512, 1};
    }
}

// Grid of a streaming form: a launch holds < 2^32 threads along x, so tiles past STREAM_GRID_X
// go on in further rows of the grid (fewer than 2^31 tiles: at most 512 rows).
constexpr int64_t STREAM_GRID_X = (int64_t)1 << 22;

struct StreamGrid {
    unsigned x, y;
};

inline StreamGrid stream_grid(int64_t tiles)
{
    const int64_t x = tiles < STREAM_GRID_X ? tiles : STREAM_GRID_X;
    return {(unsigned)x, (unsigned)((tiles + x - 1) / x)};
}

// The form for `groups` matrices of N rows and `rows` tokens each (dense: one group; experts: the
// mean). Measured with weights from HBM, f32 out, M x N x K or tokens x
// top_k x experts x N x K, us:
//  - Up to 16 rows a streaming tile of 16 x 16 per workgroup while there are at most 1024 (16 x
//    11008 x 4096 9.6, 64 x 64 tiles 10.3; 1 x 4096 x 11008 6.5, 16 x 32 10.5); beyond, up to 8
//    rows 16 x 32 with four waves (4 x 4 x 32 x 4096 x 2816 16.9 against 23.7; 16 x 2 x 8 x 11008 x
//    4096 38.4, 64 x 128 tiles 46.8), more rows the tiled forms (16 x 131072 x 4096 54 against 74).
//  - More rows: a streaming form while its workgroups fit the chip once, in the smallest tile
//    that does (64 x 4096 x 4096 in 32 x 32 7.2, tiled 64 x 64 9.2; 128 x 4096 x 4096, 512
//    workgroups, 11.5 against 9.5).
//  - 64 x 64 tiles, three stages, up to 512 of them, two to a CU (experts, whose rows are not their
//    mean, get more tiles: workgroups for half as many again, which start as others end: 512 rows of
//    4 experts, 4096 x 4096, 28.2 -> 25.5): 256 x 4096 x 4096 9.8, in 128 x
//    128 15.6; 512 x 4096 x 11008 33.9 against 46.6; 256 x 11008 x 4096 (688 tiles) 23.1 against 20.1.
//  - 64 x 128 tiles for many matrices of few rows: 128 x 2 x 8 x 11008 x 4096 (32 rows) 48.8, 128 x
//    128 54.1; 256 x 2 x 8 x 11008 x 4096 (64 rows) 69.9 against 56.5.
//  - 256 x 256 tiles (one to a CU) take about 4/3 of a round of 128 x 128 (two to a CU) at four
//    times the work of a tile: the fewer rounds, weighted so, win. 1024 x 11008 x 4096 39.0
//    against 49.3, 2048 x 4096 x 4096 32.8 against 25.8. Experts' rows are not their mean: half a
//    tile more for each. 1024 x 2 x 8 x 11008 x 4096 (256 rows) 98 against 114, 256 x 2 x 8 x 11008 x
//    4096 (64 rows) 79.5 against 56.8.
// The tiled forms' stores want N <= 2^24; wider matrices stream.
inline Form choose(int64_t groups, int64_t rows, int64_t N)
{
    auto tiles = [&](int64_t bm, int64_t bn) { return groups * ((rows + bm - 1) / bm) * ((N + bn - 1) / bn); };
    const bool tiled = N <= (1 << 24);
    if (tiles(16, 16) <= (rows <= 16 ? 1024 : 256)) return Form::S16x16;
    if (rows <= 8 || (rows <= 16 && !tiled)) return Form::S16x32;
    if (rows > 16 && tiles(32, 16) <= 256) return Form::S32x16;
    if (rows > 16 && (tiles(32, 32) <= 256 || !tiled)) return Form::S32x32;
    if (tiles(64, 64) <= 512) return Form::T64;
    if (rows <= 40) return Form::T64x128;
    auto mean_tiles = [&](int64_t b) {
        const int64_t halves = groups > 1 ? groups * (2 * rows + b) / b : 2 * ((rows + b - 1) / b);      // of row tiles
        return halves * ((N + b - 1) / b) / 2;
    };
    const int64_t r128 = (mean_tiles(128) + 511) / 512, r256 = (mean_tiles(256) + 255) / 256;
    return 3 * r128 < 4 * r256 ? Form::T128 : Form::T256;
}

// Experts: the form for the mean rows of the experts that can have any.
inline Form experts_form(int64_t rows, int64_t S, int64_t E, int64_t N, int64_t K)
{
    const int64_t used = E < S ? E : S;
    const Form form = choose(used, (S + used - 1) / used, N);
    // the tiled forms address the activations from their first row with 32 bits
    return form >= Form::T64 && rows * (K / 2) >= (int64_t)0xFFFFFF00 ? Form::S32x32 : form;
}

// Row tiles of bm rows, at most: an expert with c > 0 rows has at most 1 + (c - 1) / bm.
inline int64_t experts_row_tiles(int64_t S, int64_t E, int64_t bm)
{
    const int64_t used = E < S ? E : S;
    return used + (S - used) / bm;
}

}  // namespace qpg
