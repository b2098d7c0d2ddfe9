// gdn_attn_tc.cuh -- the tensor-memory kernel of the attention over a paged cache (bf16 caches).
#pragma once

#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

// Whether it takes the call: bf16, more rows per key head than one 16-row tile of the streaming kernel
// holds, pages of a multiple of 8 slots (a TMA copy fills whole 1024-byte atoms of the swizzled tile).
bool tc_applies(const AttnArgs& a);
// Its layout for `rows` rows per key head on `sms` SMs, and its launch.
Plan plan_tc(int sms, int rows);
cudaError_t launch_tc(const Args& x, const Plan& p, cudaStream_t stream);

}  // namespace attn
}  // namespace gdn
