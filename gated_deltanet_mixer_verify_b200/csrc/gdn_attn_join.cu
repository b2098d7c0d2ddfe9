// gdn_attn_join.cu -- adds up the parts of the rows whose positions were split over several CTAs
// (see gdn_attn.cuh for the split).
//
// With m_i, l_i, o_i the maxima, totals and sums of the parts i of a row, in base 2:
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  o = sum 2^(m_i - m) o_i / l,  lse = (m + log2 l) ln 2.
// A small grid, launched as a programmatic dependent so that it is in place when the last part is
// written. Every CTA gathers the split items from the leads that the kernel before left, and takes rows in
// turn: a warp for each row, eight parts in flight, or all its warps for one row where there are few
// rows (then each has many parts). Bound by the latency of two dependent reads:
// 4 to 7.5 us alone (148 to 296 parts of up to 48 rows), of which the launch beside the kernel before hides the start.
#include "gdn_attn.cuh"

namespace gdn {
namespace attn {
namespace {

using namespace dev;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxLeads = kMaxSms * 3;      // CTAs per row tile at most

// A row's running sums.
template <int N>
struct Sum {
    float m, l, o[N];
    bool gone;      // a part's CTA gave up
};

// 2^x, but never 0: a part's sums may be infinite (a value was), and stay so however small its weight. A part this far
// below the others adds 2^-126 of itself at most.
__device__ __forceinline__ float weight(float x) { return fmaxf(exp2_approx(x), 0x1p-126f); }

// Parts p0, p0 + step, ... below end of one row.
template <int D>
__device__ __forceinline__ void add_parts(const Args& x, const Deal& deal, int C, int tile, int r, const Lead& it, int p0, int step,
                                          int lane, Sum<D / 32>& s) {
    constexpr int N = D / 32, F = 8;
    const int c1 = it.c1_slot >> 1;
    for (int p = p0; p <= c1; p += step * F) {
        float pm[F], pl[F], po[F][N];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int cc = p + f * step;
            pm[f] = -INFINITY;
            pl[f] = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) po[f][i] = 0.f;
            // with fewer units than CTAs some have none, and left nothing
            if (cc <= c1 && deal.first(cc) < deal.first(cc + 1)) {
                const size_t at = (((size_t)tile * C + cc) * 2 + (cc == it.c0 ? (it.c1_slot & 1) : 0)) * x.rows + r;
                pm[f] = x.parts.m[at];
                pl[f] = x.parts.l[at];
#pragma unroll
                for (int i = 0; i < N; ++i) po[f][i] = x.parts.o[at * D + i * 32 + lane];
            }
        }
        float top = s.m;
#pragma unroll
        for (int f = 0; f < F; ++f) {
            s.gone |= isnan(pm[f]);
            top = fmaxf(top, pm[f]);
        }
        const float use = top == -INFINITY ? 0.f : top;
        const float k = weight(s.m - use);
        s.l *= k;
#pragma unroll
        for (int i = 0; i < N; ++i) s.o[i] *= k;
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const float w = weight(pm[f] - use);
            s.l = fmaf(w, pl[f], s.l);
#pragma unroll
            for (int i = 0; i < N; ++i) s.o[i] = fmaf(w, po[f][i], s.o[i]);
        }
        s.m = top;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) gdn_paged_attention_join_kernel(const __grid_constant__ Args x, int C, int all_rows) {
    constexpr int N = D / 32;
    __shared__ Lead s_lead[kMaxLeads];
    __shared__ int s_count[kWarps];
    __shared__ float s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
    const AttnArgs& a = x.a;
    const int G = a.Hq / a.Hk, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_wait();
    grid_release();
    const int64_t W = x.parts.units[0];
    // the split items, in the order of their leads
    int n = 0;
    for (int base = 1; base < C; base += kThreads) {
        const int c = base + threadIdx.x;
        Lead it = {-1, 0, 0, 0};
        if (c < C) it = x.parts.lead[c];
        const unsigned ballot = __ballot_sync(kFull, it.b >= 0);
        if (lane == 0) s_count[warp] = __popc(ballot);
        __syncthreads();
        int at = n + __popc(ballot & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += s_count[w];
            n += s_count[w];
        }
        if (it.b >= 0) s_lead[at] = it;
        __syncthreads();
    }
    if (n == 0) return;
    const Deal deal(W, C);
    const int64_t tasks = (int64_t)n * all_rows;
    const bool together = tasks <= gridDim.x;     // a CTA for each row
    for (int64_t i = together ? blockIdx.x : (int64_t)blockIdx.x * kWarps + warp; i < tasks; i += (int64_t)gridDim.x * (together ? 1 : kWarps)) {
        const int k = (int)(i / all_rows), row = (int)(i - (int64_t)k * all_rows);
        const Lead it = s_lead[k];
        const int tile = row / x.rows, r = row - tile * x.rows, t = row / G;
        if (t >= (a.q_len ? a.q_len[it.b] : a.T)) continue;
        Sum<N> s;
        s.m = -INFINITY;
        s.l = 0.f;
        s.gone = false;
#pragma unroll
        for (int e = 0; e < N; ++e) s.o[e] = 0.f;
        add_parts<D>(x, deal, C, tile, r, it, it.c0 + (together ? warp : 0), together ? kWarps : 1, lane, s);
        const int64_t out = ((int64_t)it.b * a.T + t) * a.Hq + (int64_t)it.h * G + (row - t * G);
        if (!together) {
            if (s.gone) continue;
            const float inv = 1.f / s.l;                         // (l = 0: o = 0)
#pragma unroll
            for (int e = 0; e < N; ++e) store_o(a, out * D + e * 32 + lane, s.l == 0.f ? 0.f : s.o[e] * inv);
            if (lane == 0 && a.lse) a.lse[out] = ((s.m == -INFINITY ? 0.f : s.m) + log2f(s.l)) * kLn2;
            continue;
        }
        // one row for each CTA: no second round, so s_o is written once
#pragma unroll
        for (int e = 0; e < N; ++e) s_o[warp][e * 32 + lane] = s.o[e];
        if (lane == 0) {
            s_m[warp] = s.gone ? NAN : s.m;
            s_l[warp] = s.l;
        }
        __syncthreads();
        float top = -INFINITY;
        bool gone = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            gone |= isnan(s_m[w]);
            top = fmaxf(top, s_m[w]);
        }
        if (gone) continue;                        // (the only row)
        const float use = top == -INFINITY ? 0.f : top;
        float sum = 0.f, f[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = weight(s_m[w] - use);
            sum = fmaf(f[w], s_l[w], sum);
        }
        const float inv = 1.f / sum;
        for (int e = threadIdx.x; e < D; e += kThreads) {
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) y = fmaf(f[w], s_o[w][e], y);
            store_o(a, out * D + e, sum == 0.f ? 0.f : y * inv);
        }
        if (threadIdx.x == 0 && a.lse) a.lse[out] = (use + log2f(sum)) * kLn2;
    }
}

template <int D>
cudaError_t launch(const Args& x, const Plan& p, cudaStream_t stream) {
    Launch l(dim3(2 * kMaxSms), kThreads, 0, stream);
    return cudaLaunchKernelEx(&l.cfg, gdn_paged_attention_join_kernel<D>, x, p.ctas, x.a.Hq / x.a.Hk * x.a.T);
}

}  // namespace

cudaError_t launch_join(const Args& x, const Plan& p, cudaStream_t stream) {
    if (p.ctas < 2) return cudaSuccess;
    return x.a.d == 64 ? launch<64>(x, p, stream) : x.a.d == 128 ? launch<128>(x, p, stream) : launch<256>(x, p, stream);
}

}  // namespace attn
}  // namespace gdn
