// linear_plan.h -- how a moe_mxfp8_linear call of given sizes is cut into
// workgroups.  Host code alone (no HIP), so that it can be looked at without
// a device.
#pragma once

#include <stdint.h>

#include "../../../include/ops/moe_ops.h"

namespace moe {

struct RowsGrid {
    int units, groups;          // weight units (rows / 16G), token groups of NT tiles
    int splits, split_chunks;   // parts of the inner axis, chunks of one
};

struct TileGrid {
    int row_blocks, tok_blocks;
    int splits, split_chunks;
};

// Tokens of linear_rows_kernel (128 x 4096 x 7168: 18.9 us, tiles 22.8; 128 x
// 7168 x 7168: 26.2 and 27.2; 192 x 7168 x 7168: 45.3 and 37.0)
constexpr int kRowsMaxTok = 128, kRowsMostTok = 1024;
constexpr int64_t kRowsMostWork = (int64_t)256 * 7168;  // workgroups times inner axis
constexpr int kMaxSplits = 8;
constexpr int kSplitTok = 8192;    // most tokens times splits (the workspace's bound)
constexpr int kCus = 256;

struct LinearPlan {
    bool rows;       // linear_rows_kernel
    int G, NT, W;
    RowsGrid grid;
    bool wide;       // 256 x 256 tiles (else 128 x 128)
    TileGrid tile;
    int splits;
};

inline LinearPlan linear_plan(int64_t T, int64_t rows, int64_t inner, int32_t activation, bool mx) {
    LinearPlan p{};
    const int tiles = (int)((T + 15) / 16), chunks = (int)(inner / 128);
    const bool gated = activation == MOE_EPI_SILU_MUL;
    // linear_rows_kernel: few tokens, and more where its largest workgroups (64 rows x 64 tokens)
    // all run at once and the work is small, so that the tiles' launches of few
    // workgroups would mostly wait (320 x 2048 x 2048: 8.3 us, tiles 19.6; 1024
    // x 1024 x 1024: 8.2 and 13.5; 256 x 4096 x 7168: 25.3 and 27.8; past the
    // bound 256 x 4096 x 16384: 51.6 and 45.8; 1000 x 512 x 16384: 36.1 and 30.7)
    const int64_t most = rows / 64 * ((T + 63) / 64);
    p.rows = T <= kRowsMaxTok || (T <= kRowsMostTok && most <= kCus && most * inner <= kRowsMostWork);
    int64_t splits = 1;
    if (!p.rows) {
        // 256 x 256 tiles, one per CU, decode each element for twice as many
        // products; 128 x 128, two per CU, lose less to a round of few tiles.
        // Up to one round of wide tiles: wide if the narrow ones would not run
        // all at once; beyond it: wide if they fill three quarters of the
        // places of their rounds (K 4096, wide and narrow, us: 140 wide tiles,
        // 504 narrow 88, 68; 144, 576 83, 86; 308, 1232 176, 153; 364, 1456 177,
        // 179; 392, 1568 181, 196; 532, 2128 279, 257; 616, 2464 279, 287; 784,
        // 3136 378, 365; 1024, 4096 408, 463)
        const int64_t wide_blocks = (rows + 255) / 256 * ((T + 255) / 256);
        const int64_t narrow_blocks = (rows + 127) / 128 * ((T + 127) / 128);
        p.wide = wide_blocks <= kCus ? narrow_blocks > 2 * kCus
                                     : 4 * wide_blocks >= 3 * ((wide_blocks + kCus - 1) / kCus * kCus);
        const int n = p.wide ? 256 : 128;
        p.tile.row_blocks = (int)((rows + n - 1) / n);
        p.tile.tok_blocks = (int)((T + n - 1) / n);
        // A 128-k chunk of a workgroup takes about 0.9 us, the pass over the
        // split sums 2 us and 0.5 us per MB of them; the number of splits that
        // leaves the least, of those that fit on the CUs (1001 x 2048 x 6144:
        // 36.6 us in 2, 46.1 in 1, 38.9 in 3; 512 x 2048 x 7168: 28.5 in 4,
        // 34.2 in 2; 1024 x 2048 x 2048: 22.5 in 2, 21.2 in 1).
        const int64_t blocks = (int64_t)p.tile.row_blocks * p.tile.tok_blocks;
        const int64_t sums = T * rows * 4 / 1000000;  // MB
        int64_t best = 9 * chunks;                    // in units of 0.1 us
        for (int64_t n = 2; !p.wide && n <= kMaxSplits && n * blocks <= kCus && n * T <= kSplitTok; n++) {
            const int64_t t = 9 * ((chunks + n - 1) / n) + 20 + 5 * n * sums;
            if (t < best) best = t, splits = n;
        }
    } else {
        // Of the tile shapes, the one whose workgroups come closest to one
        // per CU from below: fewer leave CUs idle, more take a second round
        // (and read the tokens or the weights more often).  Measured on 30
        // shapes of 9 to 128 tokens; e.g. 24 x 7168 x 7168: 224 workgroups
        // 15.3 us, 448 17.6, 112 19.3; 96 x 4096 x 7168: 256 15.1, 192 16.4,
        // 384 18.9.  Equal counts: the smaller tile.
        int64_t best = 0;
        for (int G = mx && gated ? 4 : mx || gated ? 2 : 1; G <= 4; G *= 2)
            for (int NT = 1; NT <= 4; NT++) {
                if (NT > tiles || (NT == 4 && G == 1)) continue;
                const int64_t n = rows / (16 * G) * ((tiles + NT - 1) / NT);
                const bool fits = n <= kCus, best_fits = best <= kCus;
                if (best && (fits != best_fits ? best_fits : fits ? n < best : n > best)) continue;
                if (best == n && G * NT >= p.G * p.NT) continue;
                best = n;
                p.G = G;
                p.NT = NT;
            }
        p.W = p.NT == 4 ? 4 : 8;  // what the staged tokens leave room for
        p.grid.groups = (tiles + p.NT - 1) / p.NT;
        // MXFP8 output needs whole blocks of columns in a workgroup; where
        // that leaves few of them the inner axis is split (9 x 4096 x 6144
        // gated: 64 workgroups 13.2 us, 4 times as many 11.1)
        if (mx && best <= kCus / 4) splits = 4;
    }
    if (splits > chunks / 8) splits = chunks / 8;
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (splits < 1) splits = 1;
    const int per = (int)((chunks + splits - 1) / splits);
    p.splits = (chunks + per - 1) / per;
    p.grid.splits = p.tile.splits = p.splits;
    p.grid.split_chunks = p.tile.split_chunks = per;
    if (p.rows) p.grid.units = (int)(rows / (16 * p.G));
    return p;
}

}  // namespace moe
