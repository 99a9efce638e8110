// attention_plan.h -- how a moe_tree_attention call of given sizes is cut into
// workgroups.  Host code alone (no HIP), so that it can be looked at without
// a device.
#pragma once

#include <stdint.h>

namespace moe {

// Positions that a workgroup takes at once
constexpr int kAttnUnit = 128;

struct AttentionPlan {
    int rows;            // of a workgroup: (drafted token, query head of a key/value head)
    int groups;          // workgroups, a multiple of 8
    int64_t part_floats; // floats of one partial result: the rows' elements, and two statistics a row
    int64_t bytes;       // of the workspace: two partial results per workgroup
};

inline AttentionPlan attention_plan(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t D) {
    AttentionPlan p{};
    if (T <= 0 || B <= 0) return p;
    // the rows of an average sequence (the lengths are the device's)
    const int64_t rows = (T + B - 1) / B * (heads / kv_heads);
    p.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 || D == 64 ? 64 : 128;
    p.groups = D == 256 || p.rows >= 64 ? 256 : p.rows == 16 && D == 64 ? 768 : 512;
    p.part_floats = p.rows * (D + 2);
    p.bytes = p.groups * 2 * p.part_floats * 4;
    return p;
}

// Units of all sequences together at most, T tokens of B sequences, a table
// of `positions` each
inline int64_t attention_most_units(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int rows,
                                    int64_t positions) {
    const int64_t tiles = T * (heads / kv_heads) / rows + B;
    return tiles * kv_heads * ((positions + kAttnUnit - 1) / kAttnUnit);
}

}  // namespace moe
