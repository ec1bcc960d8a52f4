// Which kernel and tile an E4M3 product takes, and the parts that its steps are split into.
#pragma once

#include <cmath>
#include <cstdint>

#include "mega_moe.h"

namespace mega_moe {

// The kernel and tile of a call, and the parts that its steps are split into.
struct ProductPlan {
    int kind, splits;
};

inline int64_t product_tiles(int m, int n, int bm, int bn) { return (int64_t)((m + bm - 1) / bm) * ((n + bn - 1) / bn); }

// What a kind takes, in us, beside the 2 of any call, with f tiles on the busiest of 256 compute units
// and s steps: f * tile + s * step for each tile, or s * alone for the last of an odd f where
// two share a compute unit (few rows: tile + f * s * (step + alone * m / 16), of b's rows and of a's).  Fitted
// (non-negative least squares of relative errors) to whole calls of 482 shapes, 326 of them with BF16 results, with operands
// that come from HBM: m in [1, 8192], k in [128, 8192] and n in [64, 18432] spread over their logarithms; m up to 128 and n
// up to 904 with k of 3840, 5632 and 8192; m and n up to 1024 with k up to 131072.  The least of the estimates is on
// average within 0.3% of the fastest of all kinds in 1, 2, 4 .. 64 parts, 10% at worst; on 74 shapes of the first sort
// that the fit has not seen 0.4% and 20%.  F32, fitted to the kinds within 30% of a shape's fastest (the stores of many
// results from a short k would bend the others): 0.3% and 5%, on 36 not seen 0.9% and 9%.
// Beside these, 128 x 64 (with and without two groups), 256 x 128 and (BF16) 128 x 256 were measured; without them the
// choice is no worse.  With F32 results Strip, Half, Tall and Long are hardly ever the fastest.
struct ProductKind {
    int rows, columns;
    float tile, step, alone;
};
enum { FEW, LOW, STRIP, DEEP, PAIR, HALF, MID, TALL, LONG, WIDE, KINDS };

inline ProductPlan product_plan(int m, int n, int k, int out_type) {
    constexpr float NEVER = INFINITY;
    static constexpr ProductKind FP8[KINDS] = {{16, 16, 1.14f, 0.069f, 0.048f},
                                               {32, 32, 2.34f, 0.113f, 0.113f},
                                               {32, 64, 2.77f, 0.162f, 0.162f},
                                               {64, 64, 2.39f, 0.234f, 0.234f},
                                               {64, 64, 1.25f, 0.210f, 0.347f},
                                               {64, 128, 3.06f, 0.334f, 0.334f},
                                               {128, 128, 2.17f, 0.546f, 0.783f},
                                               {192, 128, 3.24f, 0.630f, 0.630f},
                                               {128, 128, 2.76f, 0.455f, 0.455f},
                                               {256, 256, 4.43f, 1.145f, 1.145f}};
    static constexpr ProductKind EXACT_F32[KINDS] = {{16, 16, 0.0f, 0.113f, 0.052f},
                                                     {32, 32, 2.69f, 0.138f, 0.138f},
                                                     {32, 64, NEVER, 0.0f, 0.0f},
                                                     {64, 64, 3.26f, 0.388f, 0.388f},
                                                     {64, 64, 2.02f, 0.342f, 0.660f},
                                                     {64, 128, NEVER, 0.0f, 0.0f},
                                                     {128, 128, 3.77f, 0.985f, 1.340f},
                                                     {192, 128, NEVER, 0.0f, 0.0f},
                                                     {128, 128, NEVER, 0.0f, 0.0f},
                                                     {128, 256, 7.59f, 1.851f, 1.851f}};
    const bool f32 = out_type == MEGA_MOE_F32;
    // what parts add: a second launch, whose threads add the parts one after another, and the sums' bytes
    // (in both kernels, where BF16 results leave the first one at half of a sum's)
    constexpr float JOIN = 2.8f, JOIN_PART = 0.23f;
    const float join_element = f32 ? 0.9e-6f : 2e-6f;
    const ProductKind* kinds = f32 ? EXACT_F32 : FP8;
    const int steps = k / 128, first = m <= 16 ? FEW : LOW;
    ProductPlan best = {first, 1};
    float least = INFINITY;
    for (int kind = first; kind < KINDS; ++kind) {
        const ProductKind& o = kinds[kind];
        const int64_t tiles = product_tiles(m, n, o.rows, o.columns);
        // parts of the steps only where a compute unit would have no tile without them
        for (int splits = 1; splits == 1 || (kind != FEW && splits <= steps && tiles * splits <= 512 && splits <= 64); splits *= 2) {
            if (kind == LONG && tiles * splits > 256) break;
            const int64_t f = (tiles * splits + 255) / 256, s = (steps + splits - 1) / splits;
            float us = kind == FEW ? o.tile + f * s * (o.step + o.alone * m / 16.0f) : f * o.tile + s * ((f - f % 2) * o.step + f % 2 * o.alone);
            if (splits > 1) us += JOIN + JOIN_PART * splits + join_element * splits * (float)m * n;
            if (us < least) {
                least = us;
                best = {kind, splits};
            }
        }
    }
    return best;
}

}  // namespace mega_moe
