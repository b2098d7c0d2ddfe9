// gdn_attn_tc.cuh -- the tensor-memory kernel of the attention over a paged cache (bf16 caches).
#pragma once

#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

// Whether it takes the call. The streaming kernel is the faster one for few rows per key head (its products are
// 16 rows each, and read the cache once per 16, 32 for d <= 128) and for little work (its CTAs start sooner, two or
// three to an SM). What the lengths are is not known on the host; the tables' capacity stands for them. Measured, streaming
// against this kernel, us (4 key heads; B x positions, rows):
//   d 64:  1 x 8192, 48: 19.8, 19.6; 32 x 4096, 32: 60, 62; 32 x 4096, 48: 94, 64; 128 x 512, 48: 77, 75
//   d 128: 1 x 2048, 48: 17.0, 17.2; 1 x 4096, 48: 19.1, 17.9; 32 x 4096, 16: 59, 65; 32 x 4096, 24: 87, 69; 32 x 4096, 48: 148, 74
//   d 256: 1 x 2048, 48: 19.5, 20.6; 1 x 4096, 48: 24.3, 21.3; 1 x 4096, 16: 17.7, 19.1; 1 x 8192, 16: 24.5, 23.0;
//          32 x 512, 8: 32.5, 30.1; 32 x 4096, 8: 128, 106; 32 x 4096, 48: 346, 119
bool tc_applies(const AttnArgs& a);
// Its layout for `rows` rows per key head on `sms` SMs, and its launch.
Plan plan_tc(int sms, int rows);
cudaError_t launch_tc(const Args& x, const Plan& p, cudaStream_t stream);

}  // namespace attn
}  // namespace gdn
