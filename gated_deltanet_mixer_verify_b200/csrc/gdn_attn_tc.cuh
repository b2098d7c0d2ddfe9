// gdn_attn_tc.cuh -- the tensor-memory kernel of the attention over a paged cache (bf16 caches).
#pragma once

#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

// Its layout for `rows` rows per key head on `sms` SMs, and its launch.
Plan plan_tc(int sms, int rows);
cudaError_t launch_tc(const Args& x, const Plan& p, cudaStream_t stream);

}  // namespace attn
}  // namespace gdn
