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
    // The rows of an average sequence (the lengths are the device's), in as few
    // tiles as they fit: a tile reads and decodes its positions anew.  7 query
    // heads a key/value head, over 8000 positions, of 16 / 32 / 64 / 128 rows:
    //   32 sequences of 4 tokens (28 rows)  D 64:   69 /  52 /  69 us
    //                                       D 128: 126 /  93 / 104 us
    //                                       D 256: 295 / 186 / 229 us
    //   32 sequences of 9 tokens (63 rows)  D 64:    - /  78 /  73 us
    //                                       D 128:   - / 136 / 112 / 134 us
    //                                       D 256:   - / 345 / 249 / 308 us
    //   8 sequences of 64 tokens (448 rows) D 128:   - /   - / 157 / 149 us
    //                                       D 256:   - /   - / 413 / 339 us
    const int64_t rows = (T + B - 1) / B * (heads / kv_heads);
    p.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 || D == 64 ? 64 : 128;
    // Four waves of up to 256 registers leave room for a second workgroup a compute
    // unit; those of 64 rows and more have eight, D 256's use all registers.  Of 256
    // and 512 groups:
    //   32 sequences of 4 tokens (28 rows) over 8000   D 64:   66 /  52 us
    //                                                  D 128:  97 /  93 us
    //   64 sequences of 1 token over 8000              D 64:  107 /  83 us
    //                                                  D 128: 149 / 149 us
    //                                                  D 256: 283 / 295 us
    //   4 sequences of 1 token over 8000               D 128:  20 /  22 us
    //   1 sequence of 1 token over 30000               D 64:   16 /  17 us
    // (few sequences, whose runs are then one unit long, lose by the rule)
    p.groups = D == 256 || p.rows >= 64 ? 256 : 512;
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

// The launch that joins the parts: a wave takes one head of a token, or four
// where the rows are enough to fill the chip (one working out of the line for
// them all; 288 x 56 rows: 17 -> 9 us).  Its workgroups in rows of kJoinRow: a
// grid's dimension holds less than 2^32 threads, and 2^28 rows come to that.
constexpr int kJoinWaves = 4;  // of a workgroup
constexpr int64_t kJoinRow = 1 << 20;
struct AttentionJoin {
    int heads;      // of a wave
    unsigned x, y;  // workgroups
};

inline AttentionJoin attention_join(int64_t T, int64_t heads) {
    AttentionJoin j{};
    j.heads = T * heads >= 4096 ? 4 : 1;
    const int64_t waves = T * ((heads + j.heads - 1) / j.heads), groups = (waves + kJoinWaves - 1) / kJoinWaves;
    j.x = (unsigned)(groups < kJoinRow ? groups : kJoinRow);
    j.y = (unsigned)((groups + kJoinRow - 1) / kJoinRow);
    return j;
}

}  // namespace moe
