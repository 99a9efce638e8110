// attention_plan.h -- how a moe_tree_attention call of given sizes is cut into
// workgroups.  Host code alone (no HIP), so that it can be looked at without
// a device.
#pragma once

#include <stdint.h>

namespace moe {

// Positions that a workgroup takes at once (32 of each of its 4 waves)
constexpr int kAttnUnit = 128;

struct AttentionPlan {
    int row_tiles;       // 16-row tiles of a workgroup: rows are (drafted token, head of a kv head)
    int groups;          // workgroups
    int64_t part_floats; // floats of one partial result (16 * row_tiles rows of head_dim, and two statistics a row)
    int64_t bytes;       // of the workspace: two partial results per workgroup
};

inline AttentionPlan attention_plan(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t D) {
    AttentionPlan p{};
    if (T <= 0 || B <= 0) return p;
    // the rows of an average sequence (the lengths are the device's)
    const int64_t rows = (T + B - 1) / B * (heads / kv_heads);
    p.row_tiles = rows <= 16 ? 1 : rows <= 32 || D == 256 ? 2 : 4;
    p.groups = p.row_tiles == 4 ? 256 : 512;
    p.part_floats = (int64_t)16 * p.row_tiles * (D + 2);
    p.bytes = p.groups * 2 * p.part_floats * 4;
    return p;
}

// Units of all sequences together at most, T tokens of B sequences, a table
// of `positions` each
inline int64_t attention_most_units(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int row_tiles,
                                    int64_t positions) {
    const int64_t tiles = T * (heads / kv_heads) / (16 * row_tiles) + B;
    return tiles * kv_heads * ((positions + kAttnUnit - 1) / kAttnUnit);
}

}  // namespace moe
