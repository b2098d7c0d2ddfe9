// gdn_attn.cu -- attention of one new token or a verify block over the paged cache
// (gdn_paged_attention in include/gdn.h).
//
// One CTA per row (b, t, query head); its warps take the positions in turn, each with a running
// maximum and sum of the softmax, and are joined in shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.cuh"

namespace gdn {
namespace {

using namespace dev;

constexpr int kWarps = 4;

template <typename E, int D>
__global__ void __launch_bounds__(kWarps * 32) gdn_paged_attention_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int N = D / 32;
    __shared__ float s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kv = a.kv_len[b], q_len = a.q_len ? a.q_len[b] : a.T;
    if (kv < 0 || kv > a.max_pages * a.cache.page || q_len < 0 || q_len > a.T) {
        if (threadIdx.x == 0 && a.status_word) atomicOr(a.status_word, kStatusBadLength);
        return;
    }
    if (t >= q_len) return;
    const int p = kv - q_len + t;
    const int first = a.window > 0 ? max(0, p - a.window + 1) : 0;
    const int64_t row = ((int64_t)b * a.T + t) * a.Hq + h;
    const int64_t head = (int64_t)(h / (a.Hq / a.Hk)) * a.cache.head_stride;
    float q[N], o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = ld_in<E>(a.q, row * D + i * 32 + lane) * a.scale;
        o[i] = 0.f;
    }
    float m = -INFINITY, sum = 0.f;
    for (int j = first + warp; j <= p; j += kWarps) {
        const int id = a.table[(int64_t)b * a.max_pages + j / a.cache.page];
        if (id < 0 || id >= a.cache.num_pages) {
            if (lane == 0 && a.status_word) atomicOr(a.status_word, kStatusBadPage);
            continue;
        }
        const int64_t at = id * a.cache.page_stride + (j % a.cache.page) * a.cache.slot_stride + head;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s = fmaf(q[i], ld_in<E>(a.cache.k, at + i * 32 + lane), s);
        s = warp_sum(s);
        const float mn = fmaxf(m, s);
        const float use = mn == -INFINITY ? 0.f : mn;
        const float c = expf(m - use), w = expf(s - use);
        sum = sum * c + w;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(w, ld_in<E>(a.cache.v, at + i * 32 + lane), o[i] * c);
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s_o[warp][i * 32 + lane] = o[i];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = sum;
    }
    __syncthreads();
    float top = -INFINITY;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    const float use = top == -INFINITY ? 0.f : top;
    float l = 0.f;
    for (int w = 0; w < kWarps; ++w) l += s_l[w] * expf(s_m[w] - use);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = threadIdx.x; i < D; i += kWarps * 32) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += s_o[w][i] * expf(s_m[w] - use);
        if (a.out_bf16) st_out<__nv_bfloat16>(a.o, row * D + i, x * inv);
        else st_out<float>(a.o, row * D + i, x * inv);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[row] = use + logf(l);
}

template <typename E>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
    const dim3 grid(a.Hq, a.T, a.B);
    if (a.d == 64) gdn_paged_attention_kernel<E, 64><<<grid, kWarps * 32, 0, stream>>>(a);
    else if (a.d == 128) gdn_paged_attention_kernel<E, 128><<<grid, kWarps * 32, 0, stream>>>(a);
    else gdn_paged_attention_kernel<E, 256><<<grid, kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t paged_attention_workspace_bytes(int, int, int, int, int, bool) { return 0; }

cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t stream) {
    return a.bf16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace gdn
