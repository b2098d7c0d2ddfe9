// gdn_attn_join.cu -- adds up the parts of the rows whose positions were split over several CTAs
// (see gdn_attn.cuh for the split).
//
// With m_i, l_i, o_i the maxima, totals and sums of the parts i of a row, in base 2:
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  o = sum 2^(m_i - m) o_i / l,  lse = (m + log2 l) ln 2.
// One CTA per (border between two CTAs' units, row): the CTA of an item's first border does the
// row, all others return, so items that were not split cost nothing. Four warps take the parts
// in turn. Launched as a programmatic dependent: its CTAs are in place when the last part is written.
#include "gdn_attn.cuh"

namespace gdn {
namespace attn {
namespace {

using namespace dev;

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) gdn_paged_attention_join_kernel(const __grid_constant__ Args x, int C) {
    constexpr int N = D / 32;
    __shared__ float s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
    const AttnArgs& a = x.a;
    const int c = blockIdx.x + 1, G = a.Hq / a.Hk;
    const int tile = blockIdx.y / x.rows, r = blockIdx.y % x.rows, row = tile * x.rows + r;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (row >= G * a.T) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t W = x.parts.before[a.B];
    const int64_t u = first_unit(W, c, C);
    if (u == 0 || u >= W) return;
    // the sequence of unit u - 1 and of unit u: the last b with before[b] <= u that has units
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (x.parts.before[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    const int b = lo;
    const int64_t base = x.parts.before[b];
    const int n = (int)((x.parts.before[b + 1] - base) / a.Hk);
    const int h = (int)((u - base) / n);
    const int64_t u0 = base + (int64_t)h * n, u1 = u0 + n;
    if (u == u0) return;                                   // a border between items
    const int c0 = cta_of(W, u0, C), c1 = cta_of(W, u1 - 1, C);
    if (c != c0 + 1) return;
    const int t = row / G, q_rows = a.q_len ? a.q_len[b] : a.T;
    if (t >= q_rows) return;

    const int first_slot = first_unit(W, c0, C) == u0 ? 0 : 1;
    float m = -INFINITY, l = 0.f, o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.f;
    // eight parts in flight for each warp
    constexpr int F = 8;
    for (int p = c0 + warp; p <= c1; p += kWarps * F) {
        float pm[F], pl[F], po[F][N];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int cc = p + f * kWarps;
            pm[f] = -INFINITY;
            pl[f] = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) po[f][i] = 0.f;
            // with fewer units than CTAs some have none, and left nothing
            if (cc <= c1 && first_unit(W, cc, C) < first_unit(W, cc + 1, C)) {
                const size_t at = (((size_t)tile * C + cc) * 2 + (cc == c0 ? first_slot : 0)) * x.rows + r;
                pm[f] = x.parts.m[at];
                pl[f] = x.parts.l[at];
#pragma unroll
                for (int i = 0; i < N; ++i) po[f][i] = x.parts.o[at * D + i * 32 + lane];
            }
        }
        float top = m;
#pragma unroll
        for (int f = 0; f < F; ++f) top = fmaxf(top, pm[f]);
        const float use = top == -INFINITY ? 0.f : top;
        const float k = exp2_approx(m - use);
        l *= k;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] *= k;
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const float w = exp2_approx(pm[f] - use);
            l = fmaf(w, pl[f], l);
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = fmaf(w, po[f][i], o[i]);
        }
        m = top;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s_o[warp][i * 32 + lane] = o[i];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    const float use = top == -INFINITY ? 0.f : top;
    float sum = 0.f, k[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        k[w] = exp2_approx(s_m[w] - use);
        sum += k[w] * s_l[w];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t out = ((int64_t)b * a.T + t) * a.Hq + (int64_t)h * G + (row - t * G);
    for (int i = threadIdx.x; i < D; i += kWarps * 32) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) y = fmaf(k[w], s_o[w][i], y);
        store_o(a, out * D + i, y * inv);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[out] = (use + log2f(sum)) * kLn2;
}

template <int D>
cudaError_t launch(const Args& x, const Plan& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    const int rows = x.a.Hq / x.a.Hk * x.a.T;
    cfg.gridDim = dim3(p.ctas - 1, (rows + p.rows - 1) / p.rows * p.rows);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_paged_attention_join_kernel<D>, x, p.ctas);
}

}  // namespace

cudaError_t launch_join(const Args& x, const Plan& p, cudaStream_t stream) {
    if (p.ctas < 2) return cudaSuccess;
    return x.a.d == 64 ? launch<64>(x, p, stream) : x.a.d == 128 ? launch<128>(x, p, stream) : launch<256>(x, p, stream);
}

}  // namespace attn
}  // namespace gdn
