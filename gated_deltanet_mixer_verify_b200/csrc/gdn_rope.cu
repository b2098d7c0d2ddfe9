// gdn_rope.cu -- rotary positions with one to four axes, and the append of a block's keys and
// values to the paged cache (gdn_rope_append in include/gdn.h).
//
// Every element of q, k and v is read once and written once; the angles of a token (rot / 2 of
// them) are the same for all its heads, so a CTA forms them once in shared memory: the product
// position x frequency in fp64, reduced to a fraction of a turn there, cosine and sine in fp32.
// Bound by HBM for prompts, by latency for a block of a few tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.cuh"

namespace gdn {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

// grid (B T, ceil(rows / rows per CTA)); a row is one head of q, k or v, d / 8 lanes each hold
// eight of its elements, ITER rows per lane are in flight.
template <typename E, int D, int ITER>
__global__ void __launch_bounds__(kThreads) gdn_rope_append_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = kWarps * RPW;
    __shared__ float2 cs[D / 2];
    __shared__ int64_t s_cell;   // the slot's first element within a head's stride
    const int tok = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane % LPR;
    const int rows = a.Hq + 2 * a.Hk;
    const int r0 = blockIdx.y * (STEP * ITER) + warp * RPW + lane / LPR;

    Raw8<E> raw[ITER];
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int r = r0 + i * STEP;
        const E* p = nullptr;
        if (r < a.Hq) p = static_cast<const E*>(a.q) + (int64_t)tok * a.q_stride + (int64_t)r * D;
        else if (r < a.Hq + a.Hk) p = static_cast<const E*>(a.k) + (int64_t)tok * a.k_stride + (int64_t)(r - a.Hq) * D;
        else if (r < rows) p = static_cast<const E*>(a.v) + (int64_t)tok * a.v_stride + (int64_t)(r - a.Hq - a.Hk) * D;
        raw[i] = Raw8<E>{};
        if (p) load(p + 8 * l, raw[i]);
    }

    const int64_t slot = a.slots[tok];
    if (slot < 0) return;
    if (slot >= (int64_t)a.cache.num_pages * a.cache.page) {
        if (tid == 0 && a.status_word) atomicOr(a.status_word, kStatusBadPage);
        return;
    }
    const int half = a.rot / 2;
    for (int i = tid; i < half; i += kThreads) {
        int axis = 0;
        if (a.axes_interleaved) {
            axis = i % a.axes;
            if (i >= a.axes * a.sections[axis]) axis = 0;
        } else {
            int end = a.sections[0];
            while (i >= end) end += a.sections[++axis];   // the sections hold half pairs in all
        }
        int64_t pos;
        if (a.positions) {
            pos = a.positions[(int64_t)axis * a.B * a.T + tok];
        } else {
            const int b = tok / a.T;
            pos = (int64_t)a.kv_len[b] - a.q_len[b] + (tok - b * a.T);
        }
        // turns = pos f / 2 pi, its whole part taken off in fp64; what is left is rounded to
        // fp32 once (half a step, 2^-24 of at most half a turn: 2e-7 in angle)
        double turns = (double)pos * (double)a.inv_freq[i] * 0.15915494309189535;
        turns -= rint(turns);
        float sn, c;
        sincospif(2.f * (float)turns, &sn, &c);
        cs[i] = make_float2(c, sn);
    }
    if (tid == kThreads - 1) {
        const int64_t page = slot / a.cache.page;
        s_cell = page * a.cache.page_stride + (slot - page * a.cache.page) * a.cache.slot_stride;
    }
    __syncthreads();

#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int r = r0 + i * STEP;
        const bool is_q = r < a.Hq, is_k = !is_q && r < a.Hq + a.Hk;
        // every lane of the warp takes the shuffles, rows of v and rows past the end among them
        float x[8], y[8];
        unpack(raw[i], x);
        const float* w = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
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
        if (a.pairs_interleaved) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                y[e] = x[e];
                y[e + 1] = x[e + 1];
                if (8 * l < a.rot) {
                    const float2 t = cs[4 * l + e / 2];
                    y[e] = x[e] * t.x - x[e + 1] * t.y;
                    y[e + 1] = x[e] * t.y + x[e + 1] * t.x;
                }
            }
        } else {
            // rot / 2 is a multiple of 8: the eight partners are one lane's
            const bool first = 8 * l < half, turned = 8 * l < a.rot;
            const int other = turned ? (first ? lane + half / 8 : lane - half / 8) : lane;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = __shfl_sync(kFull, x[e], other);
                y[e] = x[e];
                if (turned) {
                    const float2 t = cs[first ? 8 * l + e : 8 * l + e - half];
                    y[e] = first ? x[e] * t.x - z * t.y : z * t.y + x[e] * t.x;
                }
            }
        }
        if (r >= rows) continue;
        if (is_q || is_k) pack(y, raw[i]);
        const int h = is_q ? r : is_k ? r - a.Hq : r - a.Hq - a.Hk;
        E* to = is_q ? static_cast<E*>(a.q_out) + (int64_t)tok * a.qo_stride + (int64_t)h * D
                     : static_cast<E*>(is_k ? a.cache.k : a.cache.v) + s_cell + h * a.cache.head_stride;
        store(to + 8 * l, raw[i]);
    }
}

template <typename E, int D>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
    constexpr int STEP = kWarps * (32 / (D / 8));
    const int rows = a.Hq + 2 * a.Hk;
    const unsigned tokens = (unsigned)a.B * (unsigned)a.T;
    // Few tokens: one row per lane, so that a token's rows spread over as many SMs as they can.
    const int per = tokens >= 148 ? (rows + STEP - 1) / STEP : 1;
    if (per <= 1)
        gdn_rope_append_kernel<E, D, 1><<<dim3(tokens, (rows + STEP - 1) / STEP), kThreads, 0, stream>>>(a);
    else if (per == 2)
        gdn_rope_append_kernel<E, D, 2><<<dim3(tokens, 1), kThreads, 0, stream>>>(a);
    else
        gdn_rope_append_kernel<E, D, 4><<<dim3(tokens, (rows + 4 * STEP - 1) / (4 * STEP)), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_d(const RopeArgs& a, cudaStream_t stream) {
    return a.d == 64 ? launch<E, 64>(a, stream) : a.d == 128 ? launch<E, 128>(a, stream) : launch<E, 256>(a, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream) {
    return a.bf16 ? launch_d<__nv_bfloat16>(a, stream) : launch_d<float>(a, stream);
}

}  // namespace gdn
