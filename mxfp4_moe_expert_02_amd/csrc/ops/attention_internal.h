// attention_internal.h -- declarations shared by the operators of
// include/ops/moe_attention.h.  Not part of the C ABI.
#pragma once

#include "../../../include/ops/moe_attention.h"
#include "attention_plan.h"
#include "ops_internal.h"

namespace moe {

// As the other operators' launchers: arguments that have passed the checks,
// every stride filled in.
hipError_t launch_kv_write(const moe_kv_rows_args& a, hipStream_t stream);
hipError_t launch_kv_read(const moe_kv_rows_args& a, hipStream_t stream);
hipError_t launch_tree_attention(const moe_tree_attention_args& a, hipStream_t stream);

}  // namespace moe
