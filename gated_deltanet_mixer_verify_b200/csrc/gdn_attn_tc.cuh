// gdn_attn_tc.cuh -- the tensor-memory kernel of the attention over a paged cache (bf16 caches).
#pragma once

#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

// Whether it takes the call. The streaming kernel is the faster one for few rows per key head (its products are
// 16 rows each, and read the cache once per 16, 32 for d <= 128) and for little work (its CTAs start sooner, two or
// three to an SM). What the lengths are is not known on the host; the tables' capacity stands for them. Measured, streaming
// against this kernel, us (4 key heads; B x positions, rows):
//   d 64:  1 x 8192, 48: 19.8, 19.6; 32 x 4096, 32: 60, 62; 48: 103, 66; 96: 149, 106; 128: 191, 118; 256: 346, 210; 128 x 512, 48: 77, 75
//   d 128: 1 x 2048, 48: 17.0, 17.2; 1 x 4096, 48: 19.1, 17.9; 32 x 4096, 16: 59, 65; 24: 87, 69; 48: 168, 72; 96: 245, 110;
//          128: 312, 125; 256: 590, 220
//   d 256: 1 x 2048, 48: 19.5, 20.6; 1 x 4096, 48: 24.3, 21.3; 1 x 4096, 16: 17.7, 19.1; 1 x 8192, 16: 24.5, 23.0;
//          32 x 512, 8: 32.5, 30.1; 32 x 4096, 8: 128, 106; 48: 399, 114; 96: 790, 155; 128: 1045, 169; 256: 2063, 298
// Other key heads (32 x 4096; key heads, rows), d 64, 128, 256: 1, 64: 35, 29; 58, 32; 144, 49; 2, 64: 60, 43; 96, 49; 271, 70; 8, 48: 187, 109;
// 308, 115; 774, 193. Where the capacity says little (48 rows), d 64, 128, 256: 32 x 4096 with a window of 128: 19.6, 20.6; 28, 21.3;
// 57, 27; of 1000: 43, 32; 70, 37; 148, 53; 32 x 300 in tables of 32,768: 25.6, 22.2; 36, 24; 68, 31; 1 x 1000 in such: 14.0, 15.8; 16.6,
// 16.0; 19.3, 20.4; 1 x 32,768 with a window of 128: 12.5, 14.6; 15.0, 15.4; 15.7, 20.1: a single short or narrow sequence loses up to
// 4 us by the rule, a batch gains.
bool tc_applies(const AttnArgs& a);
// Its layout for `rows` rows per key head on `sms` SMs, and its launch.
Plan plan_tc(int sms, int rows);
cudaError_t launch_tc(const Args& x, const Plan& p, cudaStream_t stream);

}  // namespace attn
}  // namespace gdn
