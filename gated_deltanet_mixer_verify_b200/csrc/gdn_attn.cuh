// gdn_attn.cuh -- how the attention over a paged cache is split into pieces and joined: shared by
// the streaming kernel, the tensor-memory kernel and the join kernel. Not part of the public
// interface.
//
// The lengths are on the device, so the split is made there. Every sequence b contributes, for each
// key head, an item of n_b units of `unit` positions (from the first position that any of its rows
// sees) and `extra` more that stand for the cost of an item itself. The units of a launch, ordered by
// sequence, key head and position, are dealt evenly to C CTAs, each a run of them. A CTA therefore walks whole (sequence,
// head) items, and at most its first and its last one only in part. Parts go to the workspace (two
// slots per CTA) and the join kernel adds them up in the order of the CTAs, so the result does not depend
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

// Every kernel here is launched as a programmatic dependent: it may begin while the kernel before it on
// the stream ends, waits for that one to complete before it reads or writes any global memory, and
// lets the next one begin likewise.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
struct Launch {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    Launch(dim3 grid, int threads, int smem, cudaStream_t stream) : cfg{} {
        cfg.gridDim = grid;
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

// How one launch is laid out (host).
struct Plan {
    int unit;       // positions per unit
    int extra;      // units that an item costs besides its positions
    int rows;       // rows per row tile (blockIdx.y): row r = t (H_q / H_kv) + head within the group
    int tiles;      // row tiles
    int ctas;       // CTAs per row tile (C)
    int slots() const { return ctas > 1 ? ctas * tiles * 2 : 0; }
};

// An item that was split: its sequence and key head, its first and last CTA, and the first one's slot.
// CTA c writes the entry of its own beginning: b = -1 unless it begins inside an item, and is the
// second CTA to work on it.
struct __align__(16) Lead {
    int b, h, c0, c1_slot;
};

// The workspace: the number of units and the leads, then per (row tile, CTA, slot) rows x D sums, and rows
// maxima and rows totals.
struct Parts {
    int64_t* units;   // [2], the second unused
    Lead* lead;       // [C]
    float* o;         // [tiles][C][2][rows][D]
    float* m;         // [tiles][C][2][rows], base-2 exponents (NaN: the CTA gave up)
    float* l;
};
inline size_t parts_bytes(const Plan& p, int D) {
    return p.ctas < 2 ? 0 : 16 + (size_t)p.ctas * sizeof(Lead) + (size_t)p.slots() * p.rows * ((size_t)D + 2) * 4;
}
inline Parts parts_at(void* ws, const Plan& p, int D) {
    Parts r;
    r.units = static_cast<int64_t*>(ws);
    r.lead = reinterpret_cast<Lead*>(static_cast<char*>(ws) + 16);
    r.o = reinterpret_cast<float*>(r.lead + p.ctas);
    r.m = r.o + (size_t)p.slots() * p.rows * D;
    r.l = r.m + (size_t)p.slots() * p.rows;
    return r;
}

// Arguments of the kernels.
struct Args {
    AttnArgs a;
    Parts parts;
    int rows;
    float c;        // scale log2(e): the softmax runs on base-2 exponents
    uint32_t polls; // after which a wait gives up
};
constexpr uint32_t kMaxPolls = 1u << 22;

// What a sequence asks for. rows == 0: nothing (also where its counts cannot be).
struct Seq {
    int kv, rows;   // positions, rows of the block
    int first;      // first position that any row sees
    int units;      // of an item, and with its extra ones
    int span;
};
template <int UNIT, int EXTRA>
__device__ __forceinline__ Seq make_seq(const AttnArgs& a, int kv, int rows, bool& bad) {
    Seq s;
    s.kv = kv;
    s.rows = rows;
    bad = kv < 0 || kv > a.max_pages * a.cache.page || rows < 0 || rows > a.T;
    if (bad) s.kv = s.rows = 0;
    const int p0 = s.kv - s.rows;
    s.first = a.window > 0 ? max(0, p0 - a.window + 1) / UNIT * UNIT : 0;
    s.units = s.rows == 0 ? 0 : max(1, (s.kv - s.first + UNIT - 1) / UNIT);   // a row that sees nothing is written too
    s.span = s.rows == 0 ? 0 : s.units + EXTRA;
    return s;
}
template <int UNIT, int EXTRA>
__device__ __forceinline__ Seq read_seq(const AttnArgs& a, int b, bool& bad) {
    const int kv = a.kv_len[b], rows = a.q_len ? a.q_len[b] : a.T;
    return make_seq<UNIT, EXTRA>(a, kv, rows, bad);
}

// W units dealt to C CTAs: the first W % C get one more than the others.
struct Deal {
    int64_t each, more;
    __device__ __forceinline__ Deal(int64_t W, int C) : each(W >> 32 ? W / C : (uint32_t)W / (uint32_t)C), more(W - each * C) {}
    __device__ __forceinline__ int64_t first(int c) const { return c * each + min((int64_t)c, more); }
    __device__ __forceinline__ int cta_of(int64_t u) const {
        const int64_t t = more * (each + 1);
        return (int)(u < t ? u / (each + 1) : more + (u - t) / each);
    }
};

// Where a CTA begins: its units [u, end), and the sequence that unit u falls into, whose units
// begin at `base`. All NT threads call it, with the counts of sequence threadIdx.x already asked for
// (0 rows where there is none), so that what the caller does in between hides their latency; sm holds
// NT / 32 + 2 entries. CTAs of row tile 0 leave the leads for the join.
struct Start {
    int64_t u, end, base;
    int b;
};
template <int NT, int UNIT, int EXTRA>
__device__ __forceinline__ Start find_start(const Args& x, int64_t* sm, int c, int C, int tile, int kv0, int rows0) {
    const AttnArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // NT sequences or fewer: one for each thread. More: a run of them for each.
    const int per = (a.B + NT - 1) / NT, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    bool any_bad = false;
    for (int b = b0; b < b1; ++b) {
        bool bad;
        mine += (int64_t)(per == 1 ? make_seq<UNIT, EXTRA>(a, kv0, rows0, bad) : read_seq<UNIT, EXTRA>(a, b, bad)).span * a.Hk;
        any_bad |= bad;
    }
    if (c == 0 && tile == 0 && any_bad && a.status_word) atomicOr(a.status_word, dev::kStatusBadLength);
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
    const Deal deal(W, C);
    Start s;
    s.u = deal.first(c);
    s.end = deal.first(c + 1);
    if (s.u < s.end && before <= s.u && s.u < before + mine) {
        int64_t at = before;
        int b = b0;
        bool bad;
        Seq q = read_seq<UNIT, EXTRA>(a, b, bad);
        while (s.u >= at + (int64_t)q.span * a.Hk) {
            at += (int64_t)q.span * a.Hk;
            q = read_seq<UNIT, EXTRA>(a, ++b, bad);
        }
        sm[NT / 32] = b;
        sm[NT / 32 + 1] = at;
    }
    __syncthreads();
    s.b = (int)sm[NT / 32];
    s.base = sm[NT / 32 + 1];
    if (C > 1 && tile == 0 && tid == 0) {      // behind the barrier: nobody waits for it
        Lead lead = {-1, 0, 0, 0};
        if (s.u < s.end) {
            bool bad;
            const Seq q = read_seq<UNIT, EXTRA>(a, s.b, bad);
            const int h = (int)((s.u - s.base) / q.span);
            const int64_t u0 = s.base + (int64_t)h * q.span;
            if (s.u > u0 && s.u < u0 + q.units) {
                const int c0 = deal.cta_of(u0);
                if (deal.cta_of(s.u - 1) == c0) {
                    lead.b = s.b;
                    lead.h = h;
                    lead.c0 = c0;
                    lead.c1_slot = deal.cta_of(u0 + q.units - 1) * 2 + (deal.first(c0) == u0 ? 0 : 1);
                }
            }
        }
        x.parts.lead[c] = lead;
        if (c == 0) x.parts.units[0] = W;
    }
    return s;
}
// The counts of sequence threadIdx.x, for find_start.
__device__ __forceinline__ void ask_counts(const AttnArgs& a, int& kv, int& rows) {
    kv = rows = 0;
    if ((int)threadIdx.x < a.B) {
        kv = a.kv_len[threadIdx.x];
        rows = a.q_len ? a.q_len[threadIdx.x] : a.T;
    }
}

// A CTA's walk over its items: next() moves to the next (sequence, key head) and the part of its units
// that is this CTA's. Every thread of the CTA walks alike.
template <int UNIT, int EXTRA>
struct Walk {
    int64_t u, begin, end, base;
    int b, h, i0, i1;      // sequence, key head, units i0 .. i1 of the item
    Seq s;
    bool whole;
    int slot;              // where a part goes
    __device__ __forceinline__ Walk(const Start& at) : u(at.u), begin(at.u), end(at.end), base(at.base), b(at.b) {}
    __device__ __forceinline__ bool next(const Args& x) {
        while (u < end) {
            bool bad;
            s = read_seq<UNIT, EXTRA>(x.a, b, bad);
            while (u >= base + (int64_t)s.span * x.a.Hk) {
                base += (int64_t)s.span * x.a.Hk;
                s = read_seq<UNIT, EXTRA>(x.a, ++b, bad);
            }
            const int64_t in = u - base;
            h = in >> 31 ? (int)(in / s.span) : (int)((uint32_t)in / (uint32_t)s.span);
            i0 = (int)(in - (int64_t)h * s.span);
            const int stop = (int)min((int64_t)s.span, end - u + i0);
            i1 = min(stop, s.units);
            whole = i0 == 0 && i1 == s.units;
            slot = u == begin ? 0 : 1;
            u += stop - i0;
            if (i0 < i1) return true;      // else only extra units were left of it
        }
        return false;
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

// Values that are infinite or NaN. fp32: from 2^127 (2 - 2^-11) on, where the leading tf32 term is infinite, a value is
// taken for infinite itself.
template <typename E>
__device__ __forceinline__ bool is_number(float x) { return fabsf(x) < (sizeof(E) == 4 ? 0x1.ffep127f : INFINITY); }
__device__ __forceinline__ float as_infinite(float x) { return isnan(x) ? x : copysignf(INFINITY, x); }

// The products cannot be trusted with such a value: the two terms of its weight may be zero, or of unlike signs, and zero
// times infinity or a difference of infinities is NaN. So a sum that came out NaN while its row's weights are numbers is looked up again:
// what the values of column `col` at the positions from .. to - 1 of sequence b that are no numbers add up to (0: there
// are none), every weight taken as positive. Out of line: only items that hold such values call it, eight reads at once.
template <typename E>
__device__ __noinline__ float sum_non_numbers(const AttnArgs& a, int b, int h, int col, int from, int to) {
    const int32_t* table = a.table + (int64_t)b * a.max_pages;
    const E* v = static_cast<const E*>(a.cache.v) + h * a.cache.head_stride + col;
    int page = max(from, 0) / a.cache.page, slot = max(from, 0) - page * a.cache.page;
    float sum = 0.f;
    for (int pos = max(from, 0); pos < to && !isnan(sum); pos += 8) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            y[k] = 0.f;
            if (pos + k >= to) continue;
            const int id = table[page];
            if ((unsigned)id < (unsigned)a.cache.num_pages) y[k] = dev::to_f(v[id * a.cache.page_stride + (int64_t)slot * a.cache.slot_stride]);
            if (++slot == a.cache.page) slot = 0, ++page;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (!is_number<E>(y[k])) sum += as_infinite(y[k]);
    }
    return sum;
}
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
