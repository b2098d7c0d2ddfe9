// gdn_attn_tc.cu -- attention of a verify block over the paged cache on the tensor cores (tcgen05),
// for bf16 caches and many rows per key head (see gdn_attn.cu for few rows, gdn_attn.cuh for the
// split over CTAs).
//
// With T rows per sequence and H_q / H_kv heads sharing a key head, every cached value meets T H_q /
// H_kv queries (48 for a block of 8 and 6 heads): warp matrix products in registers would be the
// bound, or the cache would have to be read once per 16 rows. Here up to 128 rows are the M of one
// tcgen05 product, so the cache is read once: S = Q K^T into tensor memory (128 x 64 positions), the
// softmax on S by one thread per row (no shuffles: a row is a tensor-memory lane), its weights back into the
// columns of S as two bf16 terms (2^-17 relative), O += P V with A from tensor memory and V as it lies
// in the cache (positions x d, N-major). O stays in tensor memory for the whole item; a row's running
// maximum only moves when it has grown by 2^8, so O is rescaled a few times per item, not per tile.
//
// One CTA per SM, ten warps with roles of their own: 0-3 softmax and outputs, 4-7 fetch keys and values
// into a ring of tiles (16-byte asynchronous copies; each warp finds the pages of its 16 of a tile's
// 64 positions, so pages of any size and any strides will do), 8 issues the products, 9 fetches
// queries. Tiles alternate K, V in the ring; S has two buffers, so the scores of the next tile are
// formed while this one's softmax runs, and the fetch runs ahead over the items' borders. Every wait
// is bounded.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn.cuh"
#include "gdn_attn_tc.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace attn {
namespace {

using namespace dev;

constexpr int kThreads = 320;
constexpr int kTile = 64;                       // positions per tile, and per unit
constexpr int kM = 128;                         // rows of a product
constexpr uint32_t kMaxPolls = 1u << 22;
constexpr float kGrow = 8.f;                    // a maximum moves when it has grown by this (base-2 exponent)
constexpr int kMaskRing = 16;                   // more tiles than the ring and the two S buffers can hold

template <int D>
struct Cfg {
    static constexpr int kSlot = kTile * D * 2;                       // bytes of a K or V tile
    static constexpr int kSlots = D == 64 ? 16 : D == 128 ? 12 : 5;
    // Tiles whose copies a fetching thread leaves in flight before it reports the oldest (96 to 128
    // KB per SM; at most kSlots - 2, so that a product never waits for a tile whose report waits for
    // the product's own slot).
    static constexpr int kAhead = D == 64 ? 12 : D == 128 ? 8 : 3;
    static constexpr int kQ = kM * D * 2;
    static constexpr int kBytes = kSlots * kSlot + kQ + 1024;         // + alignment
    static constexpr uint32_t kCols = D == 256 ? 512 : 256;           // tensor memory: S 2 x 64, O d
    static constexpr uint32_t kO = 128;
    static constexpr int kCpr = D / 8;                                // 16-byte chunks per position
    static constexpr int kLoads = 16 * kCpr / 32;                     // per lane and tile
};

struct Bars {
    uint64_t kv_full[16], kv_empty[16], s_full[2], p_full[2], pv_done[2], q_full, q_empty, o_free, drain;
};

// Byte offset of 16-byte chunk ch of row r in a tile of `rows` rows: blocks of 64 columns, 128-byte
// rows, chunks permuted by the row (the canonical 128-byte swizzle).
__device__ __forceinline__ uint32_t tile_chunk(int rows, int r, int ch) {
    return (uint32_t)((ch >> 3) * rows * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    // a source size of 0 fills the 16 bytes with zeros and reads nothing
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ bool bf16_pair_not_numbers(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// A wait that gives up when the CTA has been given up, or after kMaxPolls polls, and then gives the
// CTA up.
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, volatile int* lost) {
    for (uint32_t i = 0; i < kMaxPolls; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*lost) return false;
    }
    *lost = 1;
    return false;
}
// The same for a whole warp: its lanes agree.
__device__ __forceinline__ bool await_warp(uint64_t* bar, uint32_t parity, volatile int* lost) {
    return __all_sync(kFull, await(bar, parity, lost));
}

// grid (C, row tiles of 128).
template <int D>
__global__ void __launch_bounds__(kThreads, 1) gdn_paged_attention_tc_kernel(const __grid_constant__ Args x) {
    using G = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Bars bars;
    __shared__ int64_t s_start[kThreads / 32 + 2];
    __shared__ alignas(8) uint16_t s_mask[kMaskRing][4];      // a tile's positions that are there, 16 for each fetching warp
    __shared__ uint16_t s_partial[16][4];          // a V slot's positions that only some rows see
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_lost, s_not_numbers;
    const AttnArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = gridDim.x, c = blockIdx.x, mtile = blockIdx.y;
    // the join kernel may take its place on the SMs now; it waits for this one to end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const uint32_t raw = smem_u32(smem_raw), base_at = (raw + 1023u) & ~1023u;
    unsigned char* const tiles = smem_raw + (base_at - raw);
    const uint32_t ring_at = base_at, q_at = base_at + G::kSlots * G::kSlot;
    if (tid == 0) {
        for (int i = 0; i < G::kSlots; ++i) {
            mbar_init(&bars.kv_full[i], 4);
            mbar_init(&bars.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.s_full[i], 2);
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.pv_done[i], 2);
        }
        mbar_init(&bars.q_full, 1);
        mbar_init(&bars.q_empty, 1);
        mbar_init(&bars.o_free, 4);
        mbar_init(&bars.drain, 1);
        fence_barrier_init();
        s_lost = 0;
        s_not_numbers = 0;
    }
    if (warp == 8) {
        tc::tmem_alloc(&s_tmem, G::kCols);
        tc::tmem_relinquish();
    }
    // rows of Q that are nobody's stay zero
    for (int i = tid; i < G::kQ / 16; i += kThreads)
        reinterpret_cast<uint4*>(tiles + G::kSlots * G::kSlot)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
    const Start at = find_start<kThreads>(x, s_start, c, C, c == 0 && mtile == 0);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;

    const int share = a.Hq / a.Hk, row0 = mtile * x.rows, all_rows = share * a.T;
    const int rows = min(x.rows, all_rows - row0);
    Walk w(at);

    if (warp < 4) {
        // ---------------------------------------------------------------- softmax and outputs
        const int r = tid, row = row0 + r, t = row / share;
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const bool busy = warp * 32 < rows;          // some lane of this warp is a row
        const float cs = x.c == 0.f ? 1.f : fabsf(x.c);
        uint32_t g = 0;                              // tiles done by this CTA
        bool fine = true;
        while (fine && w.next(x)) {
            if (row0 / share >= w.s.rows) continue;
            const Sight see(a, w.s, row0, row0 + rows, share);
            const int n = w.i1 - w.i0, first = w.s.first + w.i0 * kTile;
            const int p = see.p0 + t, lo = a.window > 0 ? p - a.window + 1 : 0;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j, ++g) {
                const uint32_t buf = g & 1, parity = (g >> 1) & 1;
                if (!(fine = await_warp(&bars.s_full[buf], parity, &s_lost))) break;
                tc::fence_after_sync();
                if (busy) {
                    const uint32_t S = lanes + buf * kTile;
                    float s[2][32];
                    tc::tmem_ld32x2(S, S + 32, s[0], s[1]);
                    if (x.c <= 0.f) {                // c is folded into the exponent as |c|
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            s[0][i] = x.c < 0.f ? -s[0][i] : 0.f;
                            s[1][i] = x.c < 0.f ? -s[1][i] : 0.f;
                        }
                    }
                    const uint64_t mask = *reinterpret_cast<const volatile uint64_t*>(s_mask[g % kMaskRing]);
                    const int pos = first + j * kTile;
                    if (mask != ~0ull || pos + kTile - 1 > see.p_min || pos < see.lo_max) {
                        const int hi = p - pos, low = lo - pos;
                        uint64_t bits = hi < 0 ? 0ull : hi >= 63 ? ~0ull : (2ull << hi) - 1;
                        if (low > 0) bits = low >= 64 ? 0ull : bits & (~0ull << low);
                        bits &= mask;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!((uint32_t)bits >> i & 1)) s[0][i] = -INFINITY;
                            if (!((uint32_t)(bits >> 32) >> i & 1)) s[1][i] = -INFINITY;
                        }
                    }
                    float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 32; ++i) top4[i & 3] = fmaxf(top4[i & 3], fmaxf(s[0][i], s[1][i]));
                    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * cs;
                    const bool grew = top > m + kGrow;
                    if (__any_sync(kFull, grew)) {
                        const float k = grew ? exp2_approx(m - top) : 1.f;      // 0 the first time
                        if (grew) m = top;
                        l *= k;
                        if (j > 0) {
                            if (!(fine = await_warp(&bars.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &s_lost))) break;
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int i = 0; i < D; i += 32) {
                                float o[2][16];
                                tc::tmem_ld16x2(lanes + G::kO + i, lanes + G::kO + i + 16, o[0], o[1]);
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    o[0][e] *= k;
                                    o[1][e] *= k;
                                }
                                tc::tmem_st16_nowait(lanes + G::kO + i, o[0]);
                                tc::tmem_st16_nowait(lanes + G::kO + i + 16, o[1]);
                            }
                            tc::tmem_st_wait();
                        }
                    }
                    const float use = m == -INFINITY ? 0.f : m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    float hi[32], lw[32];            // bf16 pairs: columns of P's two terms
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int half = i >> 4, e = 2 * (i & 15);
                        const float y0 = exp2_approx(fmaf(s[half][e], cs, -use));
                        const float y1 = exp2_approx(fmaf(s[half][e + 1], cs, -use));
                        sum[i & 3] += y0 + y1;
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(y0, y1);
                        const float2 f = __bfloat1622float2(h2);
                        const __nv_bfloat162 l2 = __floats2bfloat162_rn(y0 - f.x, y1 - f.y);
                        hi[i] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h2));
                        lw[i] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&l2));
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tc::tmem_st32(S, hi);
                    tc::tmem_st32(S + 32, lw);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[buf]);
            }
            if (!fine) break;
            if (!(fine = await_warp(&bars.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &s_lost))) break;
            tc::fence_after_sync();
            if (busy) {
                const bool mine = r < rows && t < w.s.rows;
                const bool repair = s_not_numbers != 0;
                const float inv = w.whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                const int64_t out = ((int64_t)w.b * a.T + t) * a.Hq + (int64_t)w.h * share + (row - t * share);
                const size_t part = (((size_t)mtile * C + c) * 2 + w.slot) * x.rows + r;
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    float o[2][16];
                    tc::tmem_ld16x2(lanes + G::kO + i, lanes + G::kO + i + 16, o[0], o[1]);
                    if (!mine) continue;
                    if (repair) {
                        // what was taken out of the tiles (see the fetch): to the rows that see it
                        const int end = min(w.s.kv, first + n * kTile);
                        for (int pos = max(first, see.lo_min); pos < end; ++pos) {
                            if (pos >= see.lo_max && pos <= see.p_min) {
                                pos = max(pos, min(see.p_min, end - 1));   // every row sees these: nothing was taken out
                                continue;
                            }
                            if (pos > p || pos < lo) continue;
                            const int id = a.table[(int64_t)w.b * a.max_pages + pos / a.cache.page];
                            if ((unsigned)id >= (unsigned)a.cache.num_pages) continue;
                            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.cache.v) + id * a.cache.page_stride +
                                                     (int64_t)(pos % a.cache.page) * a.cache.slot_stride +
                                                     w.h * a.cache.head_stride + i;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float y = __bfloat162float(v[e]);
                                if (!isfinite(y)) o[e >> 4][e & 15] += y;
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 y = make_float4(o[e >> 4][e & 15] * inv, o[e >> 4][(e & 15) + 1] * inv,
                                                     o[e >> 4][(e & 15) + 2] * inv, o[e >> 4][(e & 15) + 3] * inv);
                        if (w.whole) store_o4(a, out * D + i + e, y);
                        else *reinterpret_cast<float4*>(x.parts.o + part * D + i + e) = y;
                    }
                }
                if (mine) {
                    if (!w.whole) {
                        x.parts.m[part] = m;
                        x.parts.l[part] = l;
                    } else if (a.lse) {
                        a.lse[out] = ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.o_free);
        }
    } else if (warp < 8) {
        // ---------------------------------------------------------------- keys and values
        const int fw = warp - 4;                     // this warp's 16 positions of a tile
        const uint32_t page = (uint32_t)a.cache.page;
        const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.cache.k);
        const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.cache.v);
        uint32_t issued = 0, told = 0, g = 0;        // tiles of the ring issued and reported, position tiles
        // Reports the oldest tile whose copies have landed. Values that are not numbers at positions
        // that some row does not see would reach it as 0 times infinity: they leave a zero, and the rows
        // that do see them get them at the end (`repair` above).
        auto tell = [&]() {
            const uint32_t slot = told % G::kSlots;
            const uint32_t partial = s_partial[slot][fw];
            if (partial) {
#pragma unroll 1
                for (int i = 0; i < G::kLoads; ++i) {
                    const int k = i * 32 + lane, pr = k / G::kCpr, ch = k - pr * G::kCpr;
                    if (!(partial >> pr & 1)) continue;
                    uint32_t* q = reinterpret_cast<uint32_t*>(tiles + slot * G::kSlot + tile_chunk(kTile, fw * 16 + pr, ch));
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t y = q[e];
                        if (bf16_pair_not_numbers(y)) {
                            s_not_numbers = 1;
                            q[e] = ((y & 0x7f80u) == 0x7f80u ? 0u : y & 0xffffu) |
                                   ((y & 0x7f800000u) == 0x7f800000u ? 0u : y & 0xffff0000u);
                        }
                    }
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.kv_full[slot]);
            ++told;
        };
        bool fine = true;
        while (fine && w.next(x)) {
            if (row0 / share >= w.s.rows) continue;
            const Sight see(a, w.s, row0, row0 + rows, share);
            const int n = w.i1 - w.i0, first = w.s.first + w.i0 * kTile + fw * 16;
            // Lanes 0 .. 15 each look one position up, a tile ahead: its page, -1 where it is not there.
            int id = -1;
            auto look_up = [&](int j) {
                const int pos = first + j * kTile + lane;
                id = -1;
                if (lane < 16 && j < n && pos < w.s.kv && pos >= see.lo_min) {
                    id = a.table[(int64_t)w.b * a.max_pages + (uint32_t)pos / page];
                    if ((unsigned)id >= (unsigned)a.cache.num_pages) {
                        if (a.status_word) atomicOr(a.status_word, kStatusBadPage);
                        id = -1;
                    }
                }
            };
            look_up(0);
            for (int j = 0; j < n; ++j, ++g) {
                const int pos = first + j * kTile + (lane & 15);
                const int64_t off = id * a.cache.page_stride + (int64_t)((uint32_t)pos % page) * a.cache.slot_stride +
                                    w.h * a.cache.head_stride;
                const uint32_t mask = __ballot_sync(kFull, id >= 0);
                const uint32_t partial = __ballot_sync(kFull, id >= 0 && (pos > see.p_min || pos < see.lo_max));
                look_up(j + 1);
                // K, then V; the offsets fit one shuffle each
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t slot = issued % G::kSlots, round = issued / G::kSlots;
                    if (!(fine = await_warp(&bars.kv_empty[slot], (round & 1) ^ 1, &s_lost))) break;
                    if (lane == 0) {
                        s_partial[slot][fw] = kv ? (uint16_t)partial : (uint16_t)0;
                        if (!kv) s_mask[g % kMaskRing][fw] = (uint16_t)mask;
                    }
                    __syncwarp();
                    const __nv_bfloat16* from = kv ? vc : kc;
                    const uint32_t to = ring_at + slot * G::kSlot;
#pragma unroll
                    for (int i = 0; i < G::kLoads; ++i) {
                        const int k = i * 32 + lane, pr = k / G::kCpr, ch = k - pr * G::kCpr;
                        const int64_t o = __shfl_sync(kFull, off, pr);
                        const bool take = mask >> pr & 1;
                        cp_async16(to + tile_chunk(kTile, fw * 16 + pr, ch), from + (take ? o + ch * 8 : 0), take);
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (++issued - told > G::kAhead) {
                        cp_async_wait<G::kAhead>();
                        tell();
                    }
                }
                if (!fine) break;
            }
        }
        cp_async_wait<0>();
        if (fine)
            while (told < issued) tell();
    } else if (warp == 8) {
        // ---------------------------------------------------------------- products
        if (lane == 0) {
            const uint32_t id_s = tc::idesc_bf16(kM, kTile, false), id_o = tc::idesc_bf16(kM, D, true);
            uint32_t g = 0, items = 0;
            bool fine = true;
            auto score = [&](uint32_t gg, bool last) -> bool {
                const uint32_t buf = gg & 1, s = 2 * gg, slot = s % G::kSlots;
                // S's columns are free once the product with the weights in them is done
                if (gg >= 2 && !await(&bars.pv_done[buf], ((gg - 2) >> 1) & 1, &s_lost)) return false;
                if (!await(&bars.kv_full[slot], (s / G::kSlots) & 1, &s_lost)) return false;
                tc::fence_after_sync();
                const uint32_t k_at = ring_at + slot * G::kSlot;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    tc::mma_bf16_ss(tmem + buf * kTile, tc::desc_kmajor_sw128(q_at + (i >> 2) * (kM * 128) + (i & 3) * 32),
                                    tc::desc_kmajor_sw128(k_at + (i >> 2) * (kTile * 128) + (i & 3) * 32), id_s, i > 0);
                tc::mma_commit(&bars.kv_empty[slot]);
                if (last) tc::mma_commit(&bars.q_empty);
                tc::mma_commit(&bars.s_full[buf]);
                mbar_arrive(&bars.s_full[buf]);      // and what this thread has seen, the tile's mask among it
                return true;
            };
            while (fine && w.next(x)) {
                if (row0 / share >= w.s.rows) continue;
                const int n = w.i1 - w.i0;
                if (!(fine = await(&bars.q_full, items & 1, &s_lost))) break;
                if (!(fine = score(g, n == 1))) break;
                for (int j = 0; j < n; ++j, ++g) {
                    if (j + 1 < n && !(fine = score(g + 1, j + 2 == n))) break;
                    const uint32_t buf = g & 1, s = 2 * g + 1, slot = s % G::kSlots;
                    if (!(fine = await(&bars.p_full[buf], (g >> 1) & 1, &s_lost))) break;
                    if (!(fine = await(&bars.kv_full[slot], (s / G::kSlots) & 1, &s_lost))) break;
                    if (j == 0 && items > 0 && !(fine = await(&bars.o_free, (items - 1) & 1, &s_lost))) break;
                    tc::fence_after_sync();
                    const uint32_t v_at = ring_at + slot * G::kSlot, P = tmem + buf * kTile;
#pragma unroll
                    for (int i = 0; i < 2 * kTile / 16; ++i)       // the leading term of P, then the other
                        tc::mma_bf16_ts(tmem + G::kO, P + i * 8, tc::desc_mnmajor_sw128(v_at + (i & 3) * 2048, kTile * 128),
                                        id_o, j > 0 || i > 0);
                    tc::mma_commit(&bars.kv_empty[slot]);
                    tc::mma_commit(&bars.pv_done[buf]);
                    mbar_arrive(&bars.pv_done[buf]);
                }
                ++items;
            }
            if (!fine) {
                // given up: let the products in flight end before the tensor memory goes
                tc::mma_commit(&bars.drain);
                for (uint32_t i = 0; i < kMaxPolls && !mbar_try_wait(&bars.drain, 0); ++i) {}
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- queries
        uint32_t items = 0;
        while (w.next(x)) {
            if (row0 / share >= w.s.rows) continue;
            if (items > 0 && !await_warp(&bars.q_empty, (items - 1) & 1, &s_lost)) break;
            for (int i = lane; i < rows * G::kCpr; i += 32) {
                const int r = i / G::kCpr, ch = i - r * G::kCpr, row = row0 + r, t = row / share;
                const int64_t qr = ((int64_t)w.b * a.T + t) * a.Hq + (int64_t)w.h * share + (row - t * share);
                cp_async16(q_at + tile_chunk(kM, r, ch), static_cast<const __nv_bfloat16*>(a.q) + qr * D + ch * 8, true);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            cp_async_wait<0>();
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.q_full);
            ++items;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 8) tc::tmem_dealloc(tmem, G::kCols);
    if (tid == 0 && s_lost && a.status_word) atomicOr(a.status_word, kStatusWaitTimeout);
}

template <int D>
cudaError_t launch(const Args& x, const Plan& p, cudaStream_t stream) {
    cudaError_t e = ensure_smem_attr<gdn_paged_attention_tc_kernel<D>>(Cfg<D>::kBytes);
    if (e != cudaSuccess) return e;
    gdn_paged_attention_tc_kernel<D><<<dim3(p.ctas, p.tiles), kThreads, Cfg<D>::kBytes, stream>>>(x);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join(x, p, stream);
}

}  // namespace

Plan plan_tc(int sms, int rows) {
    Plan p;
    p.unit = kTile;
    p.rows = std::min(rows, kM);
    p.tiles = (rows + kM - 1) / kM;
    p.ctas = std::max(1, sms / p.tiles);
    return p;
}

cudaError_t launch_tc(const Args& x, const Plan& p, cudaStream_t stream) {
    return x.a.d == 64 ? launch<64>(x, p, stream) : x.a.d == 128 ? launch<128>(x, p, stream) : launch<256>(x, p, stream);
}

}  // namespace attn
}  // namespace gdn
