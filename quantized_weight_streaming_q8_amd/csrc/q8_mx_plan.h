// q8_mx_plan.h -- which kernel and tile a product with MX4 weights, or the gated block, takes: host
// arithmetic only.
//
// Up to 16 tokens q8_mx_matmul.hip.  From 17 on the tiles that need the least time by this estimate: whole rounds
// of workgroups on the 256 CUs, each as long as a tile's step of 512 columns.  The estimate weighs the tiles
// against each other, and takes 17 tokens as 64; it is no time.  Steps in us measured on tiles that fill one round, with weights from memory, as differences between rows of 17408 and of 8704 values
// (large tiles: 10240 and 5120), estimate in brackets:
//            32 rows      64           128          160          256 x 128    256 x 256 tokens
//     MX4    0.73 (0.67)  0.95 (0.84)  1.43 (1.18)  1.94 (1.35)  2.42 (1.8)   3.75 (2.7)
//     MX6    0.81 (0.82)  0.95 (0.97)  1.52 (1.27)  1.98 (1.42)  3.19 (2.0)   4.38 (3.0)
//     MX8    1.02 (1.02)  1.31 (1.18)  1.83 (1.50)  2.30 (1.66)  3.96 (2.8)   7.50 (5.3)
// What it chooses was the shortest in each of the six comparisons below.
#pragma once

#include <stdint.h>

#include "q8ffn.h"

namespace q8 {

struct MxPlan {
    enum Way { kNarrow, kColumns, kWide } way;
    // kColumns: row groups of a wave; a tile is 32 R rows (of both projections together) x 64 tokens.
    // kWide: a tile is 256 rows x 64 times this many tokens.
    int tile;
};

// Blocks of up to 64 tokens, 32 r rows: the tokens' way to LDS and the row groups'.
constexpr float column_time(int form, int r) {
    return form == Q8_ACTS_MX4 ? 0.50f + 0.17f * r : form == Q8_ACTS_MX6 ? 0.67f + 0.15f * r : 0.86f + 0.16f * r;
}

// 256 rows x 64 rt tokens.
constexpr float wide_time(int form, int rt) {
    if (rt == 4) return form == Q8_ACTS_MX4 ? 2.7f : form == Q8_ACTS_MX6 ? 3.0f : 5.3f;
    return form == Q8_ACTS_MX4 ? 1.8f : form == Q8_ACTS_MX6 ? 2.0f : 2.8f;
}

inline int64_t mx_rounds(int64_t tiles) { return (tiles + 255) / 256; }

// N rows of each projection, two projections or one, rows quantised on their way out (in blocks of 32
// features, which needs an even number of row groups).
inline MxPlan mx_plan(int form, int64_t N, bool two, bool quantised, int64_t n_live) {
    if (n_live <= 16) return {MxPlan::kNarrow, 0};
    const int64_t groups = (((N + 15) / 16) * (two ? 2 : 1) + 1) / 2, blocks = (n_live + 63) / 64;
    const auto columns = [&](int r) {
        return (float)mx_rounds((groups + r - 1) / r * blocks) * column_time(form, r);
    };
    int r = quantised ? 2 : 1;
    for (int other : {2, 4, 5})
        if ((!quantised || other % 2 == 0) && columns(other) < columns(r)) r = other;
    // Up to 64 tokens the way of the weights bounds the time.  Above, blocks of 64 fill the chip where few large
    // tiles would not, and cost more once both fill it (7168 x 5120, MX8: 128 tokens 19 us in blocks against 35,
    // 512 tokens 44 against 41, 1024 tokens 89 against 43).
    if (n_live <= 64) return {MxPlan::kColumns, r};
    // 7168 x 5120: 1024 tokens, MX4, in 224 small tiles 30 us, in 112 large ones 44; 4099 tokens in 924 and 476 tiles,
    // MX4 117 and 90 us, MX8 170 and 159.
    const int64_t rows = (N * (two ? 2 : 1) + 255) / 256;
    const auto wide = [&](int rt) {
        return (float)mx_rounds(rows * ((n_live + 64 * rt - 1) / (64 * rt))) * wide_time(form, rt);
    };
    const int rt = wide(4) <= wide(2) ? 4 : 2;
    if (wide(rt) < columns(r)) return {MxPlan::kWide, rt};
    return {MxPlan::kColumns, r};
}

}  // namespace q8
