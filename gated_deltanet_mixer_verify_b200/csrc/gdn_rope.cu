// gdn_rope.cu -- rotary positions with one to four axes, and the append of a block's keys and
// values to the paged cache (gdn_rope_append in include/gdn.h).
//
// Every element of q, k and v is read once and written once; the angles of a token (rot / 2 of
// them) are the same for all its heads, so a CTA forms them once in shared memory: the product
// position x frequency in fp64, reduced to a fraction of a turn there, cosine and sine in fp32.
// Bound by HBM for prompts, by latency for a block of a few tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_device.cuh"
#include "gdn_internal.cuh"

namespace gdn {
namespace {

using namespace dev;

constexpr int kMaxThreads = 256;
constexpr int kManyTokens = 148 * 8;   // from here on a CTA takes four tokens

// Eight elements as stored, and as fp32.
template <typename E>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
};
template <>
struct Raw8<float> {
    float4 a, b;
};

// A plain load: q may be rotated in place, so the read-only path is not used.
__device__ __forceinline__ void load(const __nv_bfloat16* p, Raw8<__nv_bfloat16>& r) {
    r.u = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void load(const float* p, Raw8<float>& r) {
    r.a = reinterpret_cast<const float4*>(p)[0];
    r.b = reinterpret_cast<const float4*>(p)[1];
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const Raw8<__nv_bfloat16>& r) {
    *reinterpret_cast<uint4*>(p) = r.u;
}
__device__ __forceinline__ void store(float* p, const Raw8<float>& r) {
    reinterpret_cast<float4*>(p)[0] = r.a;
    reinterpret_cast<float4*>(p)[1] = r.b;
}
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw8<float>& r, float (&x)[8]) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void pack(const float (&x)[8], Raw8<__nv_bfloat16>& r) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r.u = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&x)[8], Raw8<float>& r) {
    r.a = make_float4(x[0], x[1], x[2], x[3]);
    r.b = make_float4(x[4], x[5], x[6], x[7]);
}

// grid (groups of TT tokens, groups of rows); a row is one head of q, k or v, d / 8 lanes each hold eight
// of its elements, so a lane's cosines and sines are the same for all rows of a token and stay in
// registers. The next token's rows (ITER for each lane) are in flight while this one's are worked on.
template <typename E, int D, int ITER, int TT>
__global__ void __launch_bounds__(kMaxThreads) gdn_rope_append_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    __shared__ alignas(16) float s_cos[TT][D / 2], s_sin[TT][D / 2];
    __shared__ int64_t s_cell[TT];   // the slot's first element within a head's stride, or -1
    const int tokens = a.B * a.T, tok0 = blockIdx.x * TT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane % LPR;
    const int rows = a.Hq + 2 * a.Hk, step = (blockDim.x >> 5) * RPW;
    const int r0 = blockIdx.y * (step * ITER) + warp * RPW + lane / LPR;
    const int half = a.rot / 2;

    Raw8<E> raw[2][ITER];
    auto fetch = [&](int tok, Raw8<E>(&to)[ITER]) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int r = r0 + i * step;
            const E* p = nullptr;
            if (r < a.Hq) p = static_cast<const E*>(a.q) + (int64_t)tok * a.q_stride + (int64_t)r * D;
            else if (r < a.Hq + a.Hk) p = static_cast<const E*>(a.k) + (int64_t)tok * a.k_stride + (int64_t)(r - a.Hq) * D;
            else if (r < rows) p = static_cast<const E*>(a.v) + (int64_t)tok * a.v_stride + (int64_t)(r - a.Hq - a.Hk) * D;
            to[i] = Raw8<E>{};
            if (p) load(p + 8 * l, to[i]);
        }
    };
    fetch(tok0, raw[0]);

    for (int i = tid; i < TT * half; i += blockDim.x) {
        const int tt = i / half, e = i - tt * half, tok = tok0 + tt;
        if (tok >= tokens) break;
        int axis = 0;
        if (a.axes_interleaved) {
            axis = e % a.axes;
            if (e >= a.axes * a.sections[axis]) axis = 0;
        } else {
            int end = a.sections[0];
            while (e >= end) end += a.sections[++axis];   // the sections hold half pairs in all
        }
        int64_t pos;
        if (a.positions) {
            pos = a.positions[(int64_t)axis * tokens + tok];
        } else {
            const int b = tok / a.T;
            pos = (int64_t)a.kv_len[b] - a.q_len[b] + (tok - b * a.T);
        }
        // turns = pos f / 2 pi, its whole part taken off in fp64; what is left is rounded to
        // fp32 once (half a step, 2^-24 of at most half a turn: 2e-7 in angle)
        double turns = (double)pos * (double)a.inv_freq[e] * 0.15915494309189535;
        turns -= rint(turns);
        sincospif(2.f * (float)turns, &s_sin[tt][e], &s_cos[tt][e]);
    }
    if (tid < TT) {
        int64_t cell = -1;
        if (tok0 + tid < tokens) {
            const int64_t slot = a.slots[tok0 + tid];
            const int64_t slots = (int64_t)a.cache.num_pages * a.cache.page;
            if (slot >= 0 && slot < slots) {
                const int64_t page = slots >> 32 ? slot / a.cache.page : (uint32_t)slot / (uint32_t)a.cache.page;
                cell = page * a.cache.page_stride + (slot - page * a.cache.page) * a.cache.slot_stride;
            } else if (slot >= slots && a.status_word) {
                atomicOr(a.status_word, kStatusBadPage);
            }
        }
        s_cell[tid] = cell;
    }
    __syncthreads();

#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
        const int tok = tok0 + tt;
        if (tt + 1 < TT && tok + 1 < tokens) fetch(tok + 1, raw[(tt + 1) & 1]);
        const int64_t cell = s_cell[tt];
        if (cell < 0) continue;                              // no slot: nothing of this token is written
        // this lane's eight angles' cosines and sines (interleaved: four pairs; else the first or the
        // second element of eight)
        const bool turned = 8 * l < a.rot, first = 8 * l < half;
        float cs[8], sn[8];
        const int at = !turned ? 0 : a.pairs_interleaved ? 4 * l : first ? 8 * l : 8 * l - half;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const int i = a.pairs_interleaved ? at : at + e;
            const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[tt][i]), s4 = *reinterpret_cast<const float4*>(&s_sin[tt][i]);
            cs[e] = c4.x, cs[e + 1] = c4.y, cs[e + 2] = c4.z, cs[e + 3] = c4.w;
            sn[e] = s4.x, sn[e + 1] = s4.y, sn[e + 2] = s4.z, sn[e + 3] = s4.w;
        }
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            Raw8<E>& w8 = raw[tt & 1][i];
            const int r = r0 + i * step;
            const bool is_q = r < a.Hq, is_k = !is_q && r < a.Hq + a.Hk;
            if (__any_sync(kFull, is_q || is_k)) {           // else a copy; every lane takes the shuffles
                float x[8];
                unpack(w8, x);
                const float* w = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
                if (a.q_norm || a.k_norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                    ss = group_sum<LPR>(ss);
                    if (w) {
                        const float inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
                        const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + 8 * l));
                        const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + 8 * l) + 1);
                        const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] *= inv * ww[e];
                    }
                }
                if (a.pairs_interleaved) {
                    if (turned) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float y = x[e];
                            x[e] = y * cs[e / 2] - x[e + 1] * sn[e / 2];
                            x[e + 1] = y * sn[e / 2] + x[e + 1] * cs[e / 2];
                        }
                    }
                } else {
                    // rot / 2 is a multiple of 8: the eight partners are one lane's
                    const int other = turned ? (first ? lane + half / 8 : lane - half / 8) : lane;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float z = __shfl_sync(kFull, x[e], other);
                        if (turned) x[e] = first ? x[e] * cs[e] - z * sn[e] : z * sn[e] + x[e] * cs[e];
                    }
                }
                if (is_q || is_k) pack(x, w8);
            }
            if (r >= rows) continue;
            E* to = is_q ? static_cast<E*>(a.q_out) + (int64_t)tok * a.qo_stride + (int64_t)r * D
                         : static_cast<E*>(is_k ? a.cache.k : a.cache.v) + cell + (r - a.Hq - (is_k ? 0 : a.Hk)) * a.cache.head_stride;
            store(to + 8 * l, w8);
        }
    }
}

template <typename E, int D, int ITER, int TT>
cudaError_t launch(const RopeArgs& a, int warps, int groups, cudaStream_t stream) {
    const unsigned tokens = (unsigned)a.B * (unsigned)a.T;
    gdn_rope_append_kernel<E, D, ITER, TT><<<dim3((tokens + TT - 1) / TT, groups), 32 * warps, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename E, int D>
cudaError_t launch_rows(const RopeArgs& a, cudaStream_t stream) {
    constexpr int RPW = 32 / (D / 8), kMaxWarps = kMaxThreads / 32;
    const int units = (a.Hq + 2 * a.Hk + RPW - 1) / RPW;     // warps' worth of rows per token
    const int64_t tokens = (int64_t)a.B * a.T;
    // Few tokens: one row for each lane, so that a token's rows spread over as many SMs as they can.
    if (tokens < kManyTokens) {
        const int warps = std::min(units, 4);
        return launch<E, D, 1, 1>(a, warps, (units + warps - 1) / warps, stream);
    }
    // Many: rows per lane such that a CTA's warps hold a token, or as much of it as they can.
    const int iter = std::min(4, (units + kMaxWarps - 1) / kMaxWarps);
    const int groups = (units + kMaxWarps * iter - 1) / (kMaxWarps * iter);
    const int warps = ((units + groups - 1) / groups + iter - 1) / iter;
    if (iter == 1) return launch<E, D, 1, 4>(a, warps, groups, stream);
    if (iter == 2) return launch<E, D, 2, 4>(a, warps, groups, stream);
    if (iter == 3) return launch<E, D, 3, 4>(a, warps, groups, stream);
    return launch<E, D, 4, 4>(a, warps, groups, stream);
}

template <typename E>
cudaError_t launch_d(const RopeArgs& a, cudaStream_t stream) {
    return a.d == 64 ? launch_rows<E, 64>(a, stream) : a.d == 128 ? launch_rows<E, 128>(a, stream) : launch_rows<E, 256>(a, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream) {
    return a.bf16 ? launch_d<__nv_bfloat16>(a, stream) : launch_d<float>(a, stream);
}

}  // namespace gdn
