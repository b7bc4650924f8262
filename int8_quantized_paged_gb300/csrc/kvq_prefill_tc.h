// The tensor-core prefill kernel's launcher (kvq_prefill_tc.cu).
#pragma once

#include <cuda_runtime.h>

namespace kvq {

struct PrefillArgs;

// Query rows (tokens x heads of one kv head) of a CTA.
int prefill_tc_rows(int head_dim);
// Launches one CTA per (tile, split, kv head): lc.gridDim.x of them.
cudaError_t launch_prefill_tc(cudaLaunchConfig_t& lc, int head_dim, const PrefillArgs& a);

}  // namespace kvq
