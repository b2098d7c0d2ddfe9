// gdn_rope.cu -- rotary positions with one to four axes, and the append of a block's keys and
// values to the paged cache (gdn_rope_append in include/gdn.h).
//
// Every element of q, k and v is read once and written once; the angles of a token (rot / 2 of
// them) are the same for all its heads, so a CTA forms them once in shared memory: the product
// position x frequency in fp64, reduced to a fraction of a turn there, cosine and sine in fp32.
// Measured for 24,576 tokens of 48 heads, d 128, bf16, head norms, three axes (604 MB): 128 us, 72% of
// the measured copy rate. The next token's rows are asked into L2 a token ahead (one bulk prefetch): 142 us
// without, 130 and 135 with two and four ahead, 131 with the first tokens' asked for too. That earlier form took 109 us
// without its arithmetic, 128 without the norm, no less without the cosines, so it was bound by issue and
// the latency of HBM together; 151 with 8 tokens per CTA, 167 with 4, 169 with 32. A block of a few tokens (8 x 32
// heads, d 256) takes 3.5 us, launch and three dependent reads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.cuh"

namespace gdn {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Tokens from which on a CTA takes four, and sixteen. Measured with one, four, sixteen tokens per CTA (48 heads,
// d 128, norms): 128 tokens 4.0, 8.8, 26 us; 256 6.4, 8.9, 26; 512 11.1, 9.2, 27; 4096 83, 30, 37; 6144 124, 42, 42;
// 8192 165, 53, 50; 16,384 336, 98, 85 (20 heads, d 256: 4096 86, 26, 30; 8192 171, 45, 41).
constexpr int kFour = 320, kSixteen = 6144;

// Four elements as stored, and as fp32.
template <typename E>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
    uint2 u;
};
template <>
struct Raw4<float> {
    float4 u;
};
// A plain load: q may be rotated in place, so the read-only path is not used.
template <typename E>
__device__ __forceinline__ void load(const E* p, Raw4<E>& r) {
    r.u = *reinterpret_cast<const decltype(Raw4<E>::u)*>(p);
}
template <typename E>
__device__ __forceinline__ void store(E* p, const Raw4<E>& r) {
    *reinterpret_cast<decltype(Raw4<E>::u)*>(p) = r.u;
}
__device__ __forceinline__ void unpack(const Raw4<__nv_bfloat16>& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.u.x << 16);
    x[1] = __uint_as_float(r.u.x & 0xffff0000u);
    x[2] = __uint_as_float(r.u.y << 16);
    x[3] = __uint_as_float(r.u.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const Raw4<float>& r, float (&x)[4]) {
    x[0] = r.u.x, x[1] = r.u.y, x[2] = r.u.z, x[3] = r.u.w;
}
__device__ __forceinline__ void pack(const float (&x)[4], Raw4<__nv_bfloat16>& r) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    r.u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void pack(const float (&x)[4], Raw4<float>& r) { r.u = make_float4(x[0], x[1], x[2], x[3]); }

// Asks for `bytes` (16-byte units, as the address) to be brought into L2.
__device__ __forceinline__ void ask_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// The pair (a, b) turned by an angle.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = a;
    a = x * c - b * s;
    b = x * s + b * c;
}

// The first element of a token's slot within a head's stride, or -1 where it has none.
__device__ __forceinline__ int64_t cell_of(const RopeArgs& a, int tok, bool report) {
    const int64_t slot = a.slots[tok], slots = (int64_t)a.cache.num_pages * a.cache.page;
    if (slot < 0 || slot >= slots) {
        if (slot >= slots && report && a.status_word) atomicOr(a.status_word, kStatusBadPage);
        return -1;
    }
    const int64_t page = slots >> 32 ? slot / a.cache.page : (uint32_t)slot / (uint32_t)a.cache.page;
    return page * a.cache.page_stride + (slot - page * a.cache.page) * a.cache.slot_stride;
}

// grid (groups of TT tokens, groups of heads, 1 or 3): a CTA takes q, k and v one after the other (few tokens: one
// of them), so that pointers, strides and norm are the same for all its threads. A row is one head; d / 8
// lanes hold eight of its elements each, in two quarters so chosen that the partners of a lane's elements
// are its own: elements 4 l and rot / 2 + 4 l on for halves, 8 l on for neighbouring pairs and behind rot.
// So nothing crosses lanes but the norm's sum, a lane's norm weights stay in registers for all its rows,
// and its cosines and sines for a token's. Eight warps take a token's rows, ITER for each lane, or several
// tokens' at once where a token has few.
template <typename E, int D, int ITER, int TT>
__global__ void __launch_bounds__(kThreads, 4) gdn_rope_append_kernel(const __grid_constant__ RopeArgs a, int heads_per_cta) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    __shared__ alignas(16) float s_cos[TT][D / 2], s_sin[TT][D / 2];
    __shared__ int64_t s_cell[TT];
    const int tokens = a.B * a.T, tok0 = blockIdx.x * TT, head0 = blockIdx.y * heads_per_cta;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane % LPR;
    const int half = a.rot / 2;
    const bool turned = 8 * l < a.rot, halves = turned && !a.pairs_interleaved;
    const int o1 = halves ? 4 * l : 8 * l, o2 = halves ? half + 4 * l : 8 * l + 4;   // where the quarters begin

    if (tid < TT) s_cell[tid] = tok0 + tid < tokens ? cell_of(a, tok0 + tid, blockIdx.z == 0 && head0 == 0) : -1;
    if (blockIdx.z < 2)
        for (int i = tid; i < (TT == 1 ? half : kThreads / half * half); i += kThreads) {   // pairs x tokens abreast
            const int e = i % half, t_step = kThreads / half;
            int axis = 0;
            if (a.axes_interleaved) {
                axis = e % a.axes;
                if (e >= a.axes * a.sections[axis]) axis = 0;
            } else {
                int end = a.sections[0];
                while (e >= end) end += a.sections[++axis];   // the sections hold half pairs in all
            }
            const double f = (double)a.inv_freq[e];
            for (int tt = i / half; tt < TT && tok0 + tt < tokens; tt += t_step) {
                const int tok = tok0 + tt;
                int pos;                                      // kv_len - q_len + t is below 2^30 + 2^20
                if (a.positions) {
                    pos = a.positions[(int64_t)axis * tokens + tok];
                } else {
                    const int b = tok / a.T;
                    pos = a.kv_len[b] - a.q_len[b] + (tok - b * a.T);
                }
                // turns = pos f / 2 pi, its whole part taken off in fp64; what is left is rounded to
                // fp32 once (half a step, 2^-24 of at most half a turn: 2e-7 in angle)
                double turns = (double)pos * f * 0.15915494309189535;
                turns -= rint(turns);
                sincospif(2.f * (float)turns, &s_sin[tt][e], &s_cos[tt][e]);
            }
        }
    __syncthreads();

    for (int what = blockIdx.z; what < 3; what += gridDim.z) {
        const int all_heads = what == 0 ? a.Hq : a.Hk;
        if (head0 >= all_heads) continue;
        const int heads = min(heads_per_cta, all_heads - head0);
        const int64_t stride = what == 0 ? a.q_stride : what == 1 ? a.k_stride : a.v_stride;
        const E* src = static_cast<const E*>(what == 0 ? a.q : what == 1 ? a.k : a.v) + tok0 * stride + head0 * D;
        const int64_t h_stride = what == 0 ? D : a.cache.head_stride;
        E* dst = static_cast<E*>(what == 0 ? a.q_out : what == 1 ? a.cache.k : a.cache.v) + head0 * h_stride;
        // this warp's rows: groups of RPW heads, from group on, and its tokens: from t0 on, abreast apart
        const int groups = (heads + RPW - 1) / RPW, abreast = max(1, kWarps / groups);
        const int group = groups < kWarps ? warp % groups : warp, t0 = groups < kWarps ? warp / groups : 0;
        const int h0 = group * RPW + lane / LPR;
        if (t0 >= abreast) continue;
        const float* norm = what == 0 ? a.q_norm : what == 1 ? a.k_norm : nullptr;
        float w1[4], w2[4];
        if (norm) {
            unpack(Raw4<float>{__ldg(reinterpret_cast<const float4*>(norm + o1))}, w1);
            unpack(Raw4<float>{__ldg(reinterpret_cast<const float4*>(norm + o2))}, w2);
        }
#pragma unroll 1
        for (int tt = t0; tt < TT; tt += abreast) {
            const int64_t cell = s_cell[tt];
            if (cell < 0) continue;                          // no slot: nothing of this token is written
            const E* from = src + tt * stride;
            if (TT > 1 && group == 0 && lane == 0) {         // a token ahead of the loads below
                const int ahead = tt + abreast;
                if (ahead < TT && s_cell[ahead] >= 0) ask_l2(src + ahead * stride, heads * D * (int)sizeof(E));
            }
            E* to = dst + (what == 0 ? (int64_t)(tok0 + tt) * a.qo_stride : cell);
            Raw4<E> r1[ITER], r2[ITER];
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                const int h = h0 + i * (kWarps * RPW);
                r1[i] = r2[i] = Raw4<E>{};
                if (h < heads) {
                    load(from + h * D + o1, r1[i]);
                    load(from + h * D + o2, r2[i]);
                }
            }
            if (what < 2) {                                  // rows past the end take the shuffles too
                float c[4], s[4];
                const int at = !turned ? 0 : 4 * l;          // the lane's four pairs
                unpack(Raw4<float>{*reinterpret_cast<const float4*>(&s_cos[tt][at])}, c);
                unpack(Raw4<float>{*reinterpret_cast<const float4*>(&s_sin[tt][at])}, s);
#pragma unroll
                for (int i = 0; i < ITER; ++i) {
                    if (group + i * kWarps >= groups) break;
                    float x[4], y[4];
                    unpack(r1[i], x);
                    unpack(r2[i], y);
                    if (norm) {
                        float ss = x[0] * x[0], st = y[0] * y[0];
#pragma unroll
                        for (int e = 1; e < 4; ++e) {
                            ss = fmaf(x[e], x[e], ss);
                            st = fmaf(y[e], y[e], st);
                        }
                        const float inv = rsqrtf(group_sum<LPR>(ss + st) * (1.f / D) + a.eps);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] *= inv * w1[e];
                            y[e] *= inv * w2[e];
                        }
                    }
                    if (turned) {
                        if (a.pairs_interleaved) {
                            turn(x[0], x[1], c[0], s[0]);
                            turn(x[2], x[3], c[1], s[1]);
                            turn(y[0], y[1], c[2], s[2]);
                            turn(y[2], y[3], c[3], s[3]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) turn(x[e], y[e], c[e], s[e]);
                        }
                    }
                    pack(x, r1[i]);
                    pack(y, r2[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < ITER; ++i) {
                const int h = h0 + i * (kWarps * RPW);
                if (h < heads) {
                    store(to + h * h_stride + o1, r1[i]);
                    store(to + h * h_stride + o2, r2[i]);
                }
            }
        }
    }
}

template <typename E, int D, int ITER, int TT>
cudaError_t launch(const RopeArgs& a, int heads_per_cta, cudaStream_t stream) {
    const unsigned tokens = (unsigned)a.B * (unsigned)a.T;
    const dim3 grid((tokens + TT - 1) / TT, (a.Hq + heads_per_cta - 1) / heads_per_cta, TT == 1 ? 3 : 1);
    gdn_rope_append_kernel<E, D, ITER, TT><<<grid, kThreads, 0, stream>>>(a, heads_per_cta);
    return cudaGetLastError();
}

template <typename E, int D, int TT>
cudaError_t launch_iter(const RopeArgs& a, cudaStream_t stream) {
    constexpr int STEP = kWarps * (32 / (D / 8));
    const int iter = (a.Hq + STEP - 1) / STEP;
    if (iter == 1) return launch<E, D, 1, TT>(a, STEP, stream);
    if (iter == 2) return launch<E, D, 2, TT>(a, 2 * STEP, stream);
    return launch<E, D, 3, TT>(a, 3 * STEP, stream);
}

template <typename E, int D>
cudaError_t launch_rows(const RopeArgs& a, cudaStream_t stream) {
    constexpr int RPW = 32 / (D / 8), STEP = kWarps * RPW;   // heads that eight warps hold, one for each lane
    // Few tokens: one row for each lane, so that a token's rows spread over as many SMs as they can. More:
    // as many tokens per CTA as still give every SM its four CTAs.
    const int64_t tokens = (int64_t)a.B * a.T;
    if (tokens < kFour) return launch<E, D, 1, 1>(a, STEP, stream);
    return tokens < kSixteen ? launch_iter<E, D, 4>(a, stream) : launch_iter<E, D, 16>(a, stream);
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
