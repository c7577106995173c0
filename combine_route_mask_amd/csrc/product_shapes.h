// Which tiles a product over experts takes, from what the host knows of a call.
// Plain C++: no device code.
//
// A bf16 product takes the shape that a model of the time of the busiest CU finds
// fastest, from the number of tiles on 256 CUs and of 64-deep steps.  A step takes
// a shape's workgroup `first` us alone on its CU (waits of LDS and barriers),
// `more` us of a CU's time with others, `all` us of one of 256 where all
// CUs are busy (the clock falls); a tile's beginning and end take `edge` us.
// Fitted to, and checked against, each shape's time (us, best of the four and
// the model's choice; rows x hidden x inter):
//  - products: 1023 x 2064 x 1032 gated 26.2 (64 x 64) / 26.9 (128 x 64), down
//    12.3 / 12.3 (128 x 128), through w1 23.6 / 23.6 (128 x 64); 64 x 4096 x 2048
//    down 9.3 / 9.3 (64 x 64), others 12.7, 12.8, 19; 4000 x 4096 x 1024 through w1
//    57 / 57 (256 x 256), others 117, 92, 69; 2000 rows over 16 experts x 2048 x 768
//    gated 24.5 / 24.5 (128 x 64), others 30, 31, 33;
//  - weights' gradient: 4000 rows of 2048 x 4096 66 / 66 (128 x 128), 256 x 256 85;
//    8191 rows over 8 experts of 4096 x 4096 254 / 254 (256 x 256), 128 x 128 303;
//    2000 rows over 16 of 2048 x 768 18 / 18 (128 x 128), 256 x 256 23, 64 x 64 30.
// One to three more stages for the smaller shapes change nothing where a CU has
// one workgroup and cost where it could have several.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace moe_ep {

enum Shape { kTile64, kTile128x64, kTile128, kTile256 };

struct ShapeTime {
    int channels, rows;
    float first, more, all, edge;
};

constexpr ShapeTime kShapeTimes[] = {{64, 64, 0.3f, 0.25f, 0.0f, 1.0f},
                                     {128, 64, 0.42f, 0.365f, 0.0f, 1.5f},
                                     {128, 128, 0.75f, 0.52f, 0.0f, 2.5f},
                                     {256, 256, 1.0f, 1.0f, 1.65f, 9.0f}};

// `tiles(shape)` are its tiles, `steps` those of one.
template <typename F>
inline Shape fastest_shape(float steps, F tiles)
{
    Shape best = kTile64;
    float least = 0.0f;
    for (const Shape s : {kTile64, kTile128x64, kTile128, kTile256}) {
        const ShapeTime &t = kShapeTimes[s];
        const float n = tiles(t), turns = std::ceil(n / 256.0f);
        const float step = std::max(turns > 1.0f ? turns * t.more : t.first, t.all * n / 256.0f);
        const float time = steps * step + turns * t.edge;
        if (s == kTile64 || time < least) {
            best = s;
            least = time;
        }
    }
    return best;
}

inline float tiles_of(int64_t n, int tile) { return (float)((n + tile - 1) / tile); }

// Row tiles of `rows` rows that num_rows rows over num_experts experts make.  No
// more experts than rows have one, and no more row tiles than rows are there
// (counted for every expert, the other choice's time behind the stroke, us: 4 rows
// over 64 experts of 4096 x 1024 gated 20.3 / 24.9, gated backward 21.3 / 28.3; 8
// over 128 of 2048 x 768 13.9 / 16.5; 2 over 8 of 4096 x 7168 through w1 60.7 / 85;
// the one case found the other way, 4 over 64 of 4096 x 2048 gated, 30.9 / 29.5).
// num_rows may be a sort's capacity, behind an exchange a multiple of the rows
// that exist: the host does not know those.
inline float row_tiles_of(int64_t num_rows, int num_experts, int rows)
{
    const float busy = (float)std::min<int64_t>(num_rows, num_experts);
    // ragged experts have some tiles more than experts of the average
    const float more = num_experts > 1 ? 1.1f : 1.0f;
    return std::min(more * busy * std::ceil((float)num_rows / busy / (float)rows), (float)num_rows);
}

// Rows times weights with n channels (gated: gate and up), over k.
inline Shape product_shape_of(int64_t num_rows, int num_experts, int n, int k)
{
    return fastest_shape(tiles_of(k, 64), [&](const ShapeTime &t) {
        return row_tiles_of(num_rows, num_experts, t.rows) * tiles_of(n, t.channels);
    });
}

// The weights' gradient [n][k]: every expert's is written.
inline Shape weight_grad_shape_of(int64_t num_rows, int num_experts, int n, int k)
{
    return fastest_shape(std::ceil((float)num_rows / (float)num_experts / 64.0f), [&](const ShapeTime &t) {
        return (float)num_experts * tiles_of(n, t.rows) * tiles_of(k, t.channels);
    });
}

// The product with 4-bit weights: channels and rows a workgroup, stages.
//
// Times in us, other side behind the stroke.  With at most two workgroups for
// each CU four stages of two resident ones, else three of three: 8 rows over 8 of
// 32 experts of 4096 x 7168 (512 workgroups) 27.5 / 35.8, 64 rows over 32 of
// 4096 x 2048 28.5 / 32.5, 64 over 64 of 2048 x 1024 16.7 / 19.9.  For 17 rows or
// more stages of 64 (one workgroup a CU).  Where 64 channels a workgroup leave
// CUs without one, 16 channels straight into registers: 16 rows, dense 7168 x
// 2048, 7.9 / 10.  The rows an expert are the average, which is what the host
// knows: with 16 rows a workgroup an expert of more has its weights read again
// for every 16.
enum FourBitShape { kFew, kRows16Stages4, kRows16Stages3, kRows64 };

inline FourBitShape four_bit_shape_of(int64_t num_rows, int num_experts, int n)
{
    const int64_t rows = (num_rows + num_experts - 1) / num_experts, busy = std::min<int64_t>(num_rows, num_experts);
    if (rows > 16)
        return kRows64;
    const int64_t groups = busy * (((int64_t)n + 63) / 64);
    return groups > 512 ? kRows16Stages3 : groups >= 256 ? kRows16Stages4 : kFew;
}

} // namespace moe_ep
