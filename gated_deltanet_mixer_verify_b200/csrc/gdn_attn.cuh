// gdn_attn.cuh -- how the attention over a paged cache is split into pieces and joined: shared by
// the streaming kernel, the tensor-memory kernel and the join kernel. Not part of the public
// interface.
//
// The lengths are on the device, so the split is made there. Every sequence b contributes n_b units
// of `unit` positions (from the first position that any of its rows sees) for each key head; the
// units of a launch, ordered by sequence, key head and position, are dealt evenly to C CTAs, CTA c
// taking units floor(W c / C) .. floor(W (c + 1) / C). A CTA therefore walks whole (sequence, head)
// items, and at most its first and its last one only in part. Parts go to the workspace (two slots
// per CTA) and the join kernel adds them up in the order of the CTAs, so the result does not depend
// on timing, however the lengths are spread.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.cuh"

namespace gdn {
namespace attn {

// Most SMs the workspace is laid out for; a device with more uses this many.
constexpr int kMaxSms = 160;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How one launch is laid out (host).
struct Plan {
    int unit;       // positions per unit
    int rows;       // rows per row tile (blockIdx.y): row r = t (H_q / H_kv) + head within the group
    int tiles;      // row tiles
    int ctas;       // CTAs per row tile (C)
    int slots() const { return ctas > 1 ? ctas * tiles * 2 : 0; }
};

// The workspace: the units of the sequences before b (int64 [B + 1]), then per (row tile, CTA, slot)
// rows x D sums, and rows maxima and rows totals.
struct Parts {
    int64_t* before;
    float* o;       // [tiles][C][2][rows][D]
    float* m;       // [tiles][C][2][rows], base-2 exponents
    float* l;
};
inline size_t parts_bytes(const Plan& p, int B, int D) {
    return (((size_t)B + 1) * 8 + 15) / 16 * 16 + (size_t)p.slots() * p.rows * ((size_t)D + 2) * 4;
}
inline Parts parts_at(void* ws, const Plan& p, int B, int D) {
    Parts r;
    r.before = static_cast<int64_t*>(ws);
    r.o = reinterpret_cast<float*>(static_cast<char*>(ws) + (((size_t)B + 1) * 8 + 15) / 16 * 16);
    r.m = r.o + (size_t)p.slots() * p.rows * D;
    r.l = r.m + (size_t)p.slots() * p.rows;
    return r;
}

// Arguments of the kernels.
struct Args {
    AttnArgs a;
    Parts parts;
    int rows, unit;
    float c;        // scale log2(e): the softmax runs on base-2 exponents
};

// What a sequence asks for. rows == 0: nothing (also where its counts cannot be).
struct Seq {
    int kv, rows;   // positions, rows of the block
    int first;      // first position that any row sees
    int units;
};
__device__ __forceinline__ Seq read_seq(const AttnArgs& a, int unit, int b, bool& bad) {
    Seq s;
    s.kv = a.kv_len[b];
    s.rows = a.q_len ? a.q_len[b] : a.T;
    bad = s.kv < 0 || s.kv > a.max_pages * a.cache.page || s.rows < 0 || s.rows > a.T;
    if (bad) s.kv = s.rows = 0;
    const int p0 = s.kv - s.rows;
    s.first = a.window > 0 ? max(0, p0 - a.window + 1) / unit * unit : 0;
    s.units = s.rows == 0 ? 0 : max(1, (s.kv - s.first + unit - 1) / unit);   // a row that sees nothing is written too
    return s;
}

// First unit of CTA c of C.
__device__ __forceinline__ int64_t first_unit(int64_t W, int c, int C) { return W * c / C; }
// The CTA that takes unit u.
__device__ __forceinline__ int cta_of(int64_t W, int64_t u, int C) { return (int)(((u + 1) * C + W - 1) / W) - 1; }

// Where a CTA begins: its units [u, end), and the sequence that unit u falls into, whose units
// begin at `base`. All NT threads call it; sm holds NT / 32 + 2 entries. CTA (0, 0) also leaves the
// sequences' first units for the join.
struct Start {
    int64_t u, end, base;
    int b;
};
template <int NT>
__device__ __forceinline__ Start find_start(const Args& x, int64_t* sm, int c, int C, bool write) {
    const AttnArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + NT - 1) / NT, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    bool any_bad = false;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        mine += (int64_t)read_seq(a, x.unit, b, bad).units * a.Hk;
        any_bad |= bad;
    }
    if (write && any_bad && a.status_word) atomicOr(a.status_word, dev::kStatusBadLength);
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(dev::kFull, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) sm[warp] = incl;
    __syncthreads();
    int64_t W = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sm[w];
        W += sm[w];
    }
    if (write) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
            bool bad;
            x.parts.before[b] = at;
            at += (int64_t)read_seq(a, x.unit, b, bad).units * a.Hk;
        }
        if (tid == 0) x.parts.before[a.B] = W;
    }
    Start s;
    s.u = first_unit(W, c, C);
    s.end = first_unit(W, c + 1, C);
    if (s.u < s.end && before <= s.u && s.u < before + mine) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
            bool bad;
            const int64_t n = (int64_t)read_seq(a, x.unit, b, bad).units * a.Hk;
            if (s.u < at + n) {
                sm[NT / 32] = b;
                sm[NT / 32 + 1] = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    s.b = (int)sm[NT / 32];
    s.base = sm[NT / 32 + 1];
    return s;
}

// A CTA's walk over its items: next() moves to the next (sequence, key head) and the part of its units
// that is this CTA's. Every thread of the CTA walks alike.
struct Walk {
    int64_t u, begin, end, base;
    int b, h, i0, i1;      // sequence, key head, units i0 .. i1 of the item
    Seq s;
    bool whole;
    int slot;              // where a part goes
    __device__ __forceinline__ Walk(const Start& at) : u(at.u), begin(at.u), end(at.end), base(at.base), b(at.b) {}
    __device__ __forceinline__ bool next(const Args& x) {
        if (u >= end) return false;
        bool bad;
        s = read_seq(x.a, x.unit, b, bad);
        while (u >= base + (int64_t)s.units * x.a.Hk) {
            base += (int64_t)s.units * x.a.Hk;
            s = read_seq(x.a, x.unit, ++b, bad);
        }
        h = (int)((u - base) / s.units);
        i0 = (int)(u - base - (int64_t)h * s.units);
        i1 = (int)min((int64_t)s.units, end - u + i0);
        whole = i0 == 0 && i1 == s.units;
        slot = u == begin ? 0 : 1;
        u += i1 - i0;
        return true;
    }
};

// What the rows row0 .. row1 - 1 of a sequence see (row r: positions lo .. p, both non-decreasing in
// r): every one of them sees lo_max .. p_min, none sees below lo_min.
struct Sight {
    int p0, p_min, lo_min, lo_max;
    __device__ __forceinline__ Sight(const AttnArgs& a, const Seq& s, int row0, int row1, int share) {
        p0 = s.kv - s.rows;
        p_min = p0 + row0 / share;
        lo_min = a.window > 0 ? max(0, p_min - a.window + 1) : 0;
        lo_max = a.window > 0 ? p0 + (row1 - 1) / share - a.window + 1 : 0;
    }
    // Whether some row does not see some of the n positions from pos on.
    __device__ __forceinline__ bool partial(int pos, int n) const { return pos + n - 1 > p_min || pos < lo_max; }
};

// The last word on one element of a row: weights w, their sum, and where it goes.
__device__ __forceinline__ void store_o(const AttnArgs& a, int64_t at, float x) {
    if (a.out_bf16) dev::st_out<__nv_bfloat16>(a.o, at, x);
    else dev::st_out<float>(a.o, at, x);
}
__device__ __forceinline__ void store_o4(const AttnArgs& a, int64_t at, float4 x) {
    if (a.out_bf16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
        uint2 u;
        u.x = *reinterpret_cast<const uint32_t*>(&lo);
        u.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at) = u;
    } else {
        *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at) = x;
    }
}

// Joins the parts of every item that was split (after the kernel that wrote them, on its stream).
cudaError_t launch_join(const Args& x, const Plan& p, cudaStream_t stream);

}  // namespace attn
}  // namespace gdn
