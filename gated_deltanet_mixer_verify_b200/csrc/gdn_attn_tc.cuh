// gdn_attn_tc.cuh -- the tensor-memory kernel of the attention over a paged cache (bf16 caches).
#pragma once

#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

// Whether it takes the call. The streaming kernel is the faster one for few rows per key head (its products are
// 16 rows each, and read the cache once per 16, 32 for d <= 128) and for little work (its CTAs start sooner, two or
// three to an SM). What the lengths are is not known on the host; the tables' capacity stands for them. Measured, streaming
// against this kernel, us (4 key heads; B x positions, rows):
//   d 64:  1 x 8192, 48: 20.0, 19.9; 32 x 4096, 32: 60, 61; 32 x 4096, 48: 93, 63; 128 x 512, 48: 75, 85
//   d 128: 1 x 2048, 48: 17.0, 18.6; 1 x 4096, 48: 19.6, 19.2; 32 x 4096, 16: 59, 62; 32 x 4096, 32: 90, 69; 32 x 4096, 48: 150, 74
//   d 256: 1 x 2048, 48: 19.7, 24.6; 1 x 4096, 64: 28.4, 26.3; 1 x 4096, 16: 16.7, 18.4; 1 x 8192, 16: 20.4, 20.4;
//          32 x 4096, 8: 128, 104; 32 x 4096, 48: 346, 118
bool tc_applies(const AttnArgs& a);
// Its layout for `rows` rows per key head on `sms` SMs, and its launch.
Plan plan_tc(int sms, int rows);
cudaError_t launch_tc(const Args& x, const Plan& p, cudaStream_t stream);

}  // namespace attn
}  // namespace gdn
