// gdn_attn_tc.cu -- attention of a verify block over the paged cache on the tensor cores (tcgen05),
// for bf16 caches and many rows per key head (see gdn_attn.cu for few rows, gdn_attn.cuh for the
// split over CTAs).
//
// With T rows per sequence and H_q / H_kv heads sharing a key head, every cached value meets T H_q /
// H_kv queries (48 for a block of 8 and 6 heads). Warp matrix products in registers would be the
// bound, or the cache would have to be read once per 16 rows. Here the positions are the M of the
// products and the rows their N, so nothing is multiplied for rows that are not there:
//   S^T [128 positions x N rows] = K Q^T,   O^T [d x N] += V^T P^T,
// K and V as they lie in the cache (K-major and M-major), S^T and O^T in tensor memory. A thread owns a
// position (a lane of S^T): it masks and exponentiates its N scores and leaves the weights in shared
// memory as two bf16 terms (2^-17 relative), the K x N operand of the second product. No
// maximum crosses threads in the steady state: the exponents are taken against the row maxima of the
// item's first tile, and the threads only vote whether some score has grown past them by 2^16 (fp32 and
// bf16 have the range; nothing is lost below it), which is when maxima are taken again and O rescaled.
// The sums of the weights stay with the threads until the item ends.
//
// One CTA per SM with roles for its warps: softmax and outputs (four warps for each 32 rows), two that
// fetch keys and values into a ring of [128 positions][64 columns] blocks by TMA (one copy per run
// of a page's slots, so pages of any multiple of 8 slots and any strides will do), one that issues
// the products, one that fetches queries and looks over the values at the ends of what the rows see.
// The order of products, and of the ring, is K 0, K 1, V 0, K 2, V 1, ...: scores of the next tile
// are formed before the values of this one are needed, so a block is used up as it lands, the
// softmax runs while values land, and the whole ring is copies in flight. Every wait is bounded: a CTA that gives up
// writes nothing of the items it is at, and what was split with it is not joined.
//
// Bound: HBM and the chain within a tile together. A tile of 128 positions (d 256) is 128 KB, 5,700 cycles of
// an SM's share of HBM; its 16 score and 32 output products of M 128, N 48, K 16 take 2,300 (48 each,
// bound by their reads of A from shared memory). In the steady state a tile takes 4,900 cycles where all
// SMs hold the same number of them; beside it stand the first tiles (the pages' numbers, keys, scores and values
// one after another: 20 us cold) and the ends of items (the maxima anew, the look, the output: 2 tiles).
// Measured: one sequence of 32K positions, 8 rows x 6 heads, d 256 (134 MB) 43 us; 32 of 100 .. 8192 (546 MB)
// 110 to 118 us a call, 4.6 to 5.0 TB/s, 71 to 76% of the measured copy rate.
// Steps, the first of these cases, us: rows as M, one thread per row, P in tensor memory 71; positions as M with the
// steps of a tile one after the other 68; overlapped, and the join's grid small 56; programmatic dependents 51 to 54;
// the look in rows at once, the next queries before the last look, items weighted 3 46; a loop without exits 43.
// What lies behind a sequence in its last page costs the look at up to 15 positions and the call 9% if all of it is NaN (the
// second case: 110.5 us, 120.2; d 128 77.6, 85.1; d 64 71.2, 78.2).
// Not faster: fetching with cp.async (5,600 to 9,800 cycles a tile; the proxy fence waits for copies in flight).
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

constexpr int kTile = 128;                      // positions per tile, and per unit
// Units that an item costs besides (its first and last steps overlap little). Measured with 2, 3, 4, us: one sequence of
// 32K positions (d 256, 48 rows) 47.1, 42.6, 44.2; 32 sequences of 100 .. 8192 125, 110.9, 111.3 (d 128: 88, 76.5, 68.7; d 64: 81.5,
// 71.8, 64.9).
constexpr int kExtra = 3;
constexpr int kBlock = kTile * 128;             // bytes of [128 positions][64 columns]
constexpr float kGrow = 16.f;                   // a score this far (base 2) above its row's maximum moves the maxima
constexpr int kFetch = 2;                       // warps that fetch, every other slot each
constexpr int kMaskRing = 16;                   // more tiles than the ring holds, and the one in work

constexpr int kRows = 64;                       // rows of a row tile at most
// Tiles whose products are added up in the matrix units. Those cut where they add, always towards zero, so a sum formed in them
// all along loses with every tile (128 tiles, values of one: 2.0e-5 of it); sums of kFold tiles are therefore put together
// by ordinary additions, which round, in tensor memory beside O: 1.2e-6, however long the sequence. Calls take as long with folds of
// 8, 16 and 32 tiles as with none (the second case below 110.9, 110.9, 111.0, 110.8 us). It needs half the tensor memory at d 256, which
// is why a tile has 64 rows: with 128 of them (640 threads of 96 registers that spilled, two ring slots at d 256) calls of 96 and
// 128 rows took us, 64 then 128 rows a tile: d 64 40 and 40, 47 and 50 (one sequence of 32K), 112 and 114, 112 and 124 (32 of
// 4096); d 128 44 and 45, 49 and 53; 121 and 124, 118 and 133; d 256 63 and 66, 68 and 72; 165 and 171, 158 and 177.
constexpr int kFold = 8;

// D columns of the head.
template <int D>
struct Cfg {
    static constexpr int kGroups = 2;                                 // of 128 threads and 32 rows
    static constexpr int kSoft = 128 * kGroups;                       // threads of the softmax
    static constexpr int kThreads = kSoft + 32 * (kFetch + 2);
    static constexpr int kKb = D / 64;                                // blocks of 64 columns of a K or V tile
    static constexpr int kMb = D > 128 ? D / 128 : 1;                 // M = 128 blocks of O^T
    static constexpr int kPer = kKb / kMb;                            // blocks of a ring slot: what one of them takes of V
    static constexpr int kSlot = kPer * kBlock;
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kP = kBlock;                                 // one term of P
    // buffers of P: with two, a tile's weights are written while the product before still reads its own
    static constexpr int kPb = D <= 128 ? 2 : 1;
    static constexpr int kSlots = D == 64 ? 8 : 4;
    static constexpr int kBytes = kSlots * kSlot + kQ + 2 * kPb * kP + 1024;   // + alignment
    static constexpr uint32_t kO = 2 * kRows;                         // column of O^T behind two S^T
    static constexpr uint32_t kSum = kO + kMb * kRows;                // and of the sums of the folds before
    static constexpr uint32_t kCols = kSum + kMb * kRows <= 256 ? 256 : 512;
    static constexpr int kCpr = D / 8;                                // 16-byte chunks per row of Q
};

struct Bars {
    uint64_t kv_full[8], kv_empty[8], s_full[2], p_full[2], pv_done[2], o_free, q_full, q_empty, drain;
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
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Two bf16 values, with zeros for those that are infinite or NaN.
__device__ __forceinline__ uint32_t numbers(uint32_t w) {
    return w & ~(((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u));
}
// 0 w + sum, which is NaN from the first w that is infinite or NaN on.
__device__ __forceinline__ __nv_bfloat162 taint(uint32_t w, __nv_bfloat162 sum) {
    return __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w), __floats2bfloat162_rn(0.f, 0.f), sum);
}

// Waits of a whole warp, its lanes agreeing, that give up when the CTA has been given up, or after
// `polls` polls, and then give the CTA up. First on a count in shared memory that one thread raises:
__device__ __forceinline__ void set_count(uint32_t* count, uint32_t n) {
    asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_u32(count)), "r"(n) : "memory");
}
__device__ __forceinline__ bool await_count(uint32_t* count, uint32_t want, uint32_t polls, volatile int* lost) {
    for (uint32_t i = 0; i < polls; ++i) {
        uint32_t n;
        asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(n) : "r"(smem_u32(count)) : "memory");
        if ((int32_t)(n - want) >= 0) return true;
        if (*lost) return false;
        __nanosleep(32);
    }
    *lost = 1;
    return false;
}
// and on a barrier:
__device__ __forceinline__ bool await_warp(uint64_t* bar, uint32_t parity, uint32_t polls, volatile int* lost) {
    for (uint32_t i = 0; i < polls; ++i) {
        if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(kFull, *lost)) return false;
    }
    *lost = 1;
    return false;
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " elect.sync _|p, 0xffffffff;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(r));
    return r != 0;
}
// Named barrier `id` over 128 threads: whether some thread says yes.
__device__ __forceinline__ bool any128(int id, bool yes) {
    uint32_t r;
    asm volatile(
        "{\n"
        " .reg .pred p, q;\n"
        " setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.or.pred q, %2, 128, p;\n"
        " selp.u32 %0, 1, 0, q;\n"
        "}\n"
        : "=r"(r)
        : "r"((uint32_t)yes), "r"(id)
        : "memory");
    return r != 0;
}

// The maximum (or sum) over the warp's lanes of their v[c], c = 0 .. 31, halving: left in lane c.
template <bool MAX>
__device__ __forceinline__ float reduce32(float* v, int lane) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const float send = upper ? v[i] : v[i + off], keep = upper ? v[i + off] : v[i];
            const float other = __shfl_xor_sync(kFull, send, off);
            v[i] = MAX ? fmaxf(keep, other) : keep + other;
        }
    }
    return v[0];
}

// The outputs (or parts of them) in column `col` of n rows from `row` on, as just stored, over positions first .. end - 1
// with values among them that are no numbers: what was taken out of the tiles (`repair`, see the look below) goes to the rows that
// see it, and sums that such values turned into NaN are looked up again. The first stands at the positions before
// lo_max and behind p_min, a block's length each at most; what all rows see stands between. to: where the rows
// were stored (-1: nowhere); k: what they were scaled with (0 or NaN where the sums of their weights are).
// Slow, as nothing but infinities that rows see leads to a long look: 32 sequences of 8,192 positions with infinities in all columns
// take 4.2 ms (0.15 without), with NaN 0.4. What stands between looked up once for a column instead of once for 16 rows: 2.2 ms, but
// 114 us for 110 in calls without (registers).
__device__ __noinline__ void mend(const Args& x, int b, int h, int col, int first, int end, Sight see, int share, int row, int n, bool repair, bool whole,
                                  const int64_t* to, const float* k) {
    using E = __nv_bfloat16;
    const AttnArgs& a = x.a;
    const bool half = whole && a.out_bf16;
    float* const out = whole ? static_cast<float*>(a.o) : x.parts.o;
    auto at = [&](int r) { return to[r] * a.d + col; };
    auto stored = [&](int r) { return half ? __bfloat162float(static_cast<const E*>(a.o)[at(r)]) : out[at(r)]; };
    bool lost = false;                                           // a sum is not a number though its weights are
    for (int r = 0; r < n; ++r)
        if (to[r] >= 0 && k[r] >= 0.f) lost |= isnan(stored(r));
    if (!lost && !repair) return;
    const float all = lost ? sum_non_numbers<E>(a, b, h, col, max(first, see.lo_max), min(end, see.p_min + 1)) : 0.f;
    for (int r = 0; r < n; ++r) {
        if (to[r] < 0 || !(k[r] >= 0.f)) continue;
        const int p = see.p0 + (row + r) / share;
        const int from = max(first, a.window > 0 ? p - a.window + 1 : 0), stop = min(end, p + 1);
        const float y = sum_non_numbers<E>(a, b, h, col, from, min(stop, see.lo_max)) +
                        sum_non_numbers<E>(a, b, h, col, max(from, max(see.lo_max, see.p_min + 1)), stop);
        float o = stored(r);
        if (k[r] == 0.f) o = 0.f;
        else if (!isnan(o)) o += y;
        else if (y + all != 0.f) o = y + all;
        if (half) static_cast<E*>(a.o)[at(r)] = __float2bfloat16_rn(o);
        else out[at(r)] = o;
    }
}

// grid (C, row tiles). run: slots per copy, the largest power of two up to a tile that
// divides the page size.
template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
gdn_paged_attention_tc_kernel(const __grid_constant__ Args x, const __grid_constant__ CUtensorMap k_map,
                              const __grid_constant__ CUtensorMap v_map, int run) {
    using G = Cfg<D>;
    constexpr int kSoftWarps = G::kSoft / 32;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Bars bars;
    __shared__ int64_t s_start[G::kThreads / 32 + 2];
    __shared__ uint32_t s_mask[kMaskRing][4];      // a tile's positions that are there
    __shared__ float s_part[G::kGroups][4][32];    // per warp: maxima or sums of its positions
    __shared__ alignas(16) float s_m[G::kGroups][32];  // maxima (read four at a time)
    __shared__ alignas(16) float s_use[G::kGroups][32], s_k[G::kGroups][32];   // the same, 0 for none; factors
    __shared__ int64_t s_row[G::kGroups][32];      // where a row goes (-1: nowhere)
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_lost;
    __shared__ volatile int s_not_numbers;         // the last item with values that some row sees taken out of its tiles
    __shared__ uint32_t s_ask, s_looked;           // V tiles to be looked over, and looked over (counts)
    const AttnArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = gridDim.x, c = blockIdx.x, mtile = blockIdx.y;
    const uint32_t raw = smem_u32(smem_raw), ring_at = (raw + 1023u) & ~1023u;
    unsigned char* const ring = smem_raw + (ring_at - raw);
    constexpr uint32_t kQOff = G::kSlots * G::kSlot, kPOff = kQOff + G::kQ;
    if (tid == 0) {
        tc::prefetch_tmap(&k_map);
        tc::prefetch_tmap(&v_map);
        for (int i = 0; i < G::kSlots; ++i) {
            mbar_init(&bars.kv_full[i], 1);
            mbar_init(&bars.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.s_full[i], 2);
            mbar_init(&bars.p_full[i], kSoftWarps);
            mbar_init(&bars.pv_done[i], 2);
        }
        mbar_init(&bars.o_free, kSoftWarps);
        mbar_init(&bars.q_full, 1);
        mbar_init(&bars.q_empty, 1);
        mbar_init(&bars.drain, 1);
        fence_barrier_init();
        s_lost = 0;
        s_not_numbers = 0;
        s_ask = s_looked = 0;
    }
    if (warp == kSoftWarps + kFetch) {
        tc::tmem_alloc(&s_tmem, G::kCols);
        tc::tmem_relinquish();
    }
    // rows of Q that are nobody's stay zero
    for (int i = tid; i < G::kQ / 16; i += G::kThreads) reinterpret_cast<uint4*>(ring + kQOff)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
    // So far nothing was read that another kernel writes: this may run while the kernel before ends. The
    // join kernel may take its place on the SMs from here on; it waits for this one to end.
    grid_wait();
    grid_release();
    int kv0, rows0;
    ask_counts(a, kv0, rows0);
    const Start at = find_start<G::kThreads, kTile, kExtra>(x, s_start, c, C, mtile, kv0, rows0);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;

    const int share = a.Hq / a.Hk, row0 = mtile * x.rows, all_rows = share * a.T;
    const int rows = min(x.rows, all_rows - row0);
    Walk<kTile, kExtra> w(at);
    uint32_t issued = 0;                             // slots of the ring, as far as a fetching warp has come

    if (warp < kSoftWarps) {
        // ---------------------------------------------------------------- softmax and outputs
        const int wg = warp >> 2, k = tid & 127, bar = 1 + wg;
        const int my_rows = min(32, rows - 32 * wg);             // rows of this group of warps (not positive: none)
        const int chunks = (max(my_rows, 0) + 15) / 16;          // 16 columns each
        const int my_row0 = row0 + 32 * wg;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float cs = x.c == 0.f ? 1.f : fabsf(x.c);
        // the product of tile t is done
        auto product_done = [&](uint32_t t) { return await_warp(&bars.pv_done[t & 1], (t >> 1) & 1, x.polls, &s_lost); };
        // Tiles done by this CTA. Its first item begins with a tile -1, worked without waiting for anything and
        // forgotten: while the first keys are on their way, it brings the instructions in (4,000 cycles of misses).
        uint32_t g = ~0u;
        // The four warps of a group meet at barriers that nothing bounds. So one whose wait has given up goes on without
        // waiting, to the vote at the item's end, where all four leave or none.
        bool fine = true;
        int item = 0;                                            // counted from 1
        float l[32];
        while (fine && w.next(x)) {
            if (row0 / share >= w.s.rows) continue;
            ++item;
            const Sight see(a, w.s, row0, row0 + rows, share);
            const int n = w.i1 - w.i0, first = w.s.first + w.i0 * kTile;
            for (int j = g == ~0u ? -1 : 0; j < n; ++j, ++g) {
                if (j <= 0) {
#pragma unroll
                    for (int r = 0; r < 32; ++r) l[r] = 0.f;
                }
                if (j >= 0) fine = fine && await_warp(&bars.s_full[g & 1], (g >> 1) & 1, x.polls, &s_lost);
                tc::fence_after_sync();
                float s[32];
                if (chunks > 0) {
                    const uint32_t S = lanes + (g & 1) * kRows + 32 * wg;
                    tc::tmem_ld16x2(S, S + 16, *reinterpret_cast<float(*)[16]>(s), *reinterpret_cast<float(*)[16]>(s + 16));
                    if (x.c <= 0.f) {                            // c enters the exponents as |c|
#pragma unroll
                        for (int r = 0; r < 32; ++r) s[r] = x.c < 0.f ? -s[r] : s[r] * 0.f;
                    }
                    const int pos = first + j * kTile + k;
                    const uint32_t mask = *const_cast<const volatile uint32_t*>(&s_mask[g % kMaskRing][warp & 3]);
                    if (mask != ~0u || see.partial(first + j * kTile, kTile)) {
                        // this position is seen by the rows from .. to - 1: row r stands at p0 + r / share
                        const int64_t from = (int64_t)max(0, pos - see.p0) * share - my_row0;
                        const int64_t to = !(mask >> lane & 1) ? from : a.window > 0 ? ((int64_t)pos - see.p0 + a.window) * share - my_row0 : 32;
                        const int f = (int)max((int64_t)-1, min(from, (int64_t)32)), e = (int)max((int64_t)-1, min(to, (int64_t)32));
#pragma unroll
                        for (int r = 0; r < 32; ++r)
                            if (r < f || r >= e) s[r] = -INFINITY;
                    }
                    bool move = j <= 0;
                    if (j > 0) {
                        float over = -INFINITY;
#pragma unroll
                        for (int r = 0; r < 32; r += 4) {
                            if (r >= 16 && chunks < 2) break;
                            const float4 m = *reinterpret_cast<const float4*>(&s_m[wg][r]);
                            over = fmaxf(over, fmaxf(fmaxf(fmaf(s[r], cs, -m.x), fmaf(s[r + 1], cs, -m.y)),
                                                     fmaxf(fmaf(s[r + 2], cs, -m.z), fmaf(s[r + 3], cs, -m.w))));
                        }
                        move = any128(bar, over > kGrow);
                    }
                    if (move) {
                        float top[32];
#pragma unroll
                        for (int r = 0; r < 32; ++r) top[r] = s[r];
                        s_part[wg][warp & 3][lane] = reduce32<true>(top, lane);
                        named_barrier_sync(bar, 128);
                        if (k < 32) {
                            float m = fmaxf(fmaxf(s_part[wg][0][k], s_part[wg][1][k]), fmaxf(s_part[wg][2][k], s_part[wg][3][k])) * cs;
                            if (j > 0) {
                                const float old = s_m[wg][k];
                                m = fmaxf(m, old);
                                s_k[wg][k] = m == old ? 1.f : exp2_approx(old - m);
                            }
                            s_m[wg][k] = m;
                            s_use[wg][k] = m == -INFINITY ? 0.f : m;
                        }
                        named_barrier_sync(bar, 128);
                    }
                    // the product that last read this buffer of P; and O is rescaled behind the one before
                    if (j >= G::kPb) fine = fine && product_done(g - G::kPb);
                    if (move && j > 0) {
                        fine = fine && product_done(g - 1);
                        tc::fence_after_sync();
#pragma unroll
                        for (int r = 0; r < 32; ++r) l[r] *= s_k[wg][r];
#pragma unroll 1
                        for (int i = 0; i < G::kMb * (j > kFold ? 4 : 2); ++i) {   // O, and the sums of the folds before
                            const uint32_t O = lanes + G::kO + (i >> 1) * kRows + 32 * wg + (i & 1) * 16;
                            float o[16];
                            tc::tmem_ld16(O, o);
#pragma unroll
                            for (int r = 0; r < 16; ++r) o[r] *= s_k[wg][(i & 1) * 16 + r];
                            tc::tmem_st16_nowait(O, o);
                        }
                        tc::tmem_st_wait();
                    }
                    unsigned char* P = ring + kPOff + g % G::kPb * (2 * G::kP);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {                // eight rows: one 16-byte chunk of each term
                        if (q >= 2 * chunks) break;
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 8 * q + 2 * e;
                            const float2 m = *reinterpret_cast<const float2*>(&s_use[wg][r]);
                            const float y0 = exp2_approx(fmaf(s[r], cs, -m.x)), y1 = exp2_approx(fmaf(s[r + 1], cs, -m.y));
                            l[r] += y0;
                            l[r + 1] += y1;
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(y0, y1);
                            const float2 f = __bfloat1622float2(h2);
                            const __nv_bfloat162 l2 = __floats2bfloat162_rn(y0 - f.x, y1 - f.y);
                            hi[e] = *reinterpret_cast<const uint32_t*>(&h2);
                            lo[e] = *reinterpret_cast<const uint32_t*>(&l2);
                        }
                        const uint32_t to_chunk = tile_chunk(kTile, k, wg * 4 + q);
                        *reinterpret_cast<uint4*>(P + to_chunk) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(P + G::kP + to_chunk) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    // A fold: O is added to the sums of the folds before, and the next product begins it anew. Here, where the
                    // scores are used up (registers).
                    if (j > 0 && j % kFold == 0) {
                        fine = fine && product_done(g - 1);
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int i = 0; i < G::kMb * 2; ++i) {
                            const uint32_t O = lanes + G::kO + (i >> 1) * kRows + 32 * wg + (i & 1) * 16, sums = O + (G::kSum - G::kO);
                            float o[16], t[16];
                            tc::tmem_ld16x2(O, sums, o, t);
#pragma unroll
                            for (int r = 0; r < 16; ++r) o[r] += j > kFold ? t[r] : 0.f;
                            tc::tmem_st16_nowait(sums, o);
                        }
                        tc::tmem_st_wait();
                    }
                    tc::fence_proxy_async_smem();
                } else if (j >= G::kPb) {
                    fine = fine && product_done(g - G::kPb);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0 && j >= 0 && fine) mbar_arrive(&bars.p_full[g & 1]);
            }
            // the sums, and where the rows go
            if (chunks > 0) s_part[wg][warp & 3][lane] = reduce32<false>(l, lane);
            fine = fine && product_done(g - 1);
            if (chunks > 0) fine = !any128(bar, !fine);
            if (!fine) break;
            tc::fence_after_sync();
            if (chunks > 0) {
                if (k < 32) {
                    const int row = my_row0 + k, t = row / share;
                    const float sum = (s_part[wg][0][k] + s_part[wg][1][k]) + (s_part[wg][2][k] + s_part[wg][3][k]);
                    int64_t to = -1;
                    if (k < my_rows && t < w.s.rows) {
                        if (w.whole) {
                            to = ((int64_t)w.b * a.T + t) * a.Hq + (int64_t)w.h * share + (row - t * share);
                            if (a.lse) a.lse[to] = (s_use[wg][k] + log2f(sum)) * kLn2;
                        } else {
                            to = (((int64_t)mtile * C + c) * 2 + w.slot) * x.rows + 32 * wg + k;
                            x.parts.m[to] = isnan(s_m[wg][k]) ? -INFINITY : s_m[wg][k];   // (sum is NaN then)
                            x.parts.l[to] = sum;
                        }
                    }
                    s_row[wg][k] = to;
                    s_k[wg][k] = isnan(sum) ? sum : !w.whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                }
                named_barrier_sync(bar, 128);
                const bool repair = s_not_numbers == item;
                const int end = min(w.s.kv, first + n * kTile);
#pragma unroll 1
                for (int i = 0; i < G::kMb * chunks; ++i) {
                    const int mb = i / chunks, q = i - mb * chunks, col = mb * 128 + k;
                    const uint32_t O = lanes + G::kO + mb * kRows + 32 * wg + q * 16;
                    float o[16], t[16];
                    tc::tmem_ld16x2(O, O + (G::kSum - G::kO), o, t);
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[r] += n > kFold ? t[r] : 0.f;
                    if (col >= D) continue;                      // d = 64: the upper lanes hold it twice
                    int64_t to[16];
                    float f[16];
                    float odd[4] = {};                           // NaN if one of them is no number
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        to[r] = s_row[wg][q * 16 + r] < 0 ? -1 : s_row[wg][q * 16 + r] * D + col;
                        f[r] = o[r] * s_k[wg][q * 16 + r];
                        odd[r & 3] = fmaf(f[r], 0.f, odd[r & 3]);
                    }
                    if (!w.whole || !a.out_bf16) {
                        float* out = w.whole ? static_cast<float*>(a.o) : x.parts.o;
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (to[r] >= 0) out[to[r]] = f[r];
                    } else {
                        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o);
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (to[r] >= 0) out[to[r]] = __float2bfloat16_rn(f[r]);
                    }
                    if (repair || isnan((odd[0] + odd[1]) + (odd[2] + odd[3])))
                        mend(x, w.b, w.h, col, first, end, see, share, my_row0 + q * 16, min(16, my_rows - q * 16), repair, w.whole,
                             &s_row[wg][q * 16], &s_k[wg][q * 16]);
                }
                named_barrier_sync(bar, 128);                    // s_row, s_k and s_part are the next item's
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.o_free);
        }
    } else if (warp < kSoftWarps + kFetch) {
        // ---------------------------------------------------------------- keys and values
        // Two warps, because a lane that issues a copy takes 75 to 150 cycles for it, and a tile of short
        // pages is many copies.
        const uint32_t fw = warp - kSoftWarps;
        const int page = a.cache.page, runs = kTile / run;
        const int r = lane % runs, blk = lane / runs;            // this lane's run of the tile, and its block of a slot
        uint32_t g = 0;                              // tiles
        bool fine = true;
        while (fine && w.next(x)) {
            if (row0 / share >= w.s.rows) continue;
            const Sight see(a, w.s, row0, row0 + rows, share);
            const int n = w.i1 - w.i0, first = w.s.first + w.i0 * kTile;
            // A lane looks up the page of its run of tile j, and makes it num_pages (which TMA reads as zeros)
            // where nothing of the run is seen or the page is not in the pool.
            auto needed = [&](int j) -> bool {
                const int pos = first + j * kTile + r * run;
                return j < n && pos < w.s.kv && pos + run > see.lo_min;
            };
            auto look_up = [&](int j) -> int {
                return needed(j) ? a.table[(int64_t)w.b * a.max_pages + (first + j * kTile + r * run) / page] : 0;
            };
            auto page_of = [&](int j, int id) -> int {
                const bool need = needed(j);
                if (need && (unsigned)id < (unsigned)a.cache.num_pages) return id;
                if (need && a.status_word) atomicOr(a.status_word, kStatusBadPage);
                return a.cache.num_pages;
            };
            auto fetch = [&](const CUtensorMap* map, int j, int id, bool keys) -> bool {
                const int slot0 = (first + j * kTile + r * run) % page;
#pragma unroll 1
                for (int i = 0; i < G::kMb; ++i, ++issued) {
                    if (issued % kFetch != fw) continue;
                    const uint32_t slot = issued % G::kSlots, round = issued / G::kSlots;
                    if (!await_warp(&bars.kv_empty[slot], (round & 1) ^ 1, x.polls, &s_lost)) return false;
                    if (keys && i == 0) {
                        // the tile's positions that are there, 32 to a word
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int bit = r * run - 32 * q;                // this lane's run within the word
                            uint32_t bits = 0;
                            if (id < a.cache.num_pages && bit < 32 && bit + run > 0)
                                bits = run >= 32 ? ~0u : ((1u << run) - 1) << bit;
                            bits = __reduce_or_sync(kFull, bits);
                            if (lane == 0) s_mask[g % kMaskRing][q] = bits;
                        }
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&bars.kv_full[slot], G::kSlot);
                    __syncwarp();
                    if (blk < G::kPer)
                        tc::tma_load_4d(ring + slot * G::kSlot + blk * kBlock + r * run * 128, map, (i * G::kPer + blk) * 64, w.h, slot0, id,
                                        &bars.kv_full[slot]);
                }
                return true;
            };
            // K 0, K 1, V 0, K 2, V 1, ...; pages are looked up a tile ahead of their use
            int id_v = 0, id_k = look_up(0), id_next = look_up(1);
            for (int j = 0; j <= n; ++j) {
                if (j < n) {
                    id_k = page_of(j, id_k);
                    if (!(fine = fetch(&k_map, j, id_k, true))) break;
                    ++g;
                }
                if (j > 0 && !(fine = fetch(&v_map, j - 1, id_v, false))) break;
                id_v = id_k;
                id_k = id_next;
                id_next = look_up(j + 2);
            }
        }
    } else if (warp == kSoftWarps + kFetch) {
        // ---------------------------------------------------------------- products
        // The whole warp walks and waits alike and one elected lane issues: what the products take (addresses,
        // descriptors) is then the same in every lane by construction, and a run of products differs by
        // constants only: 48 cycles each, where descriptors made one by one, or in a lane's own branch, cost
        // 80 to 140. A wait costs 150 more, so there is one for each slot of the ring.
        const uint32_t tm = __shfl_sync(kFull, tmem, 0);
        const uint32_t N = (uint32_t)(rows + 15) / 16 * 16;
        const uint32_t id_s = tc::idesc_bf16(kTile, N, false), id_o = tc::idesc_bf16(128, N, true);
        uint32_t g = 0, items = 0, looked = 0;
        uint32_t slot = 0, phase = 0;                            // of the ring: the next one
        const uint64_t q_at = tc::desc_kmajor_sw128(ring_at + kQOff), p_base = tc::desc_mnmajor_sw128(ring_at + kPOff, kBlock);
        bool fine = true;
        while (fine && w.next(x)) {
            if (row0 / share >= w.s.rows) continue;
            const Sight see(a, w.s, row0, row0 + rows, share);
            const int n = __shfl_sync(kFull, w.i1 - w.i0, 0), first = __shfl_sync(kFull, w.s.first + w.i0 * kTile, 0);
            if (!(fine = await_warp(&bars.q_full, items & 1, x.polls, &s_lost))) break;
            // S^T = K Q^T of tile j: into the buffer that tile j - 2's reader has left
            auto score = [&](int j) -> bool {
                const uint32_t buf = (g + j) & 1;
#pragma unroll
                for (int mb = 0; mb < G::kMb; ++mb) {
                    if (!await_warp(&bars.kv_full[slot], phase, x.polls, &s_lost)) return false;
                    tc::fence_after_sync();
                    if (elect_one()) {
                        const uint64_t k_at = tc::desc_kmajor_sw128(ring_at + slot * G::kSlot);
#pragma unroll
                        for (int i = 0; i < 4 * G::kPer; ++i)
                            tc::mma_bf16_ss(tm + buf * kRows, k_at + ((i >> 2) * kBlock + (i & 3) * 32) / 16,
                                            q_at + ((mb * G::kPer + (i >> 2)) * (kRows * 128) + (i & 3) * 32) / 16, id_s, mb > 0 || i > 0);
                        tc::mma_commit(&bars.kv_empty[slot]);
                        if (mb == G::kMb - 1) {
                            if (j == n - 1) tc::mma_commit(&bars.q_empty);
                            tc::mma_commit(&bars.s_full[buf]);
                            mbar_arrive(&bars.s_full[buf]);      // and what this warp has seen, the tile's mask among it
                        }
                    }
                    __syncwarp();
                    if (++slot == G::kSlots) slot = 0, phase ^= 1;
                }
                return true;
            };
            if (!(fine = score(0))) break;
            for (int j = 0; j < n; ++j) {
                if (j + 1 < n && !(fine = score(j + 1))) break;
                // O^T += V^T P^T
                if (!(fine = await_warp(&bars.p_full[(g + j) & 1], ((g + j) >> 1) & 1, x.polls, &s_lost))) break;
                if (j == 0 && items > 0 && !(fine = await_warp(&bars.o_free, (items - 1) & 1, x.polls, &s_lost))) break;
                if (see.partial(first + j * kTile, kTile)) {
                    uint32_t sl = slot, ph = phase;
                    for (int mb = 0; mb < G::kMb && fine; ++mb) {
                        fine = await_warp(&bars.kv_full[sl], ph, x.polls, &s_lost);
                        if (++sl == G::kSlots) sl = 0, ph ^= 1;
                    }
                    if (!fine) break;
                    ++looked;
                    if (lane == 0) set_count(&s_ask, looked);
                    if (!(fine = __all_sync(kFull, await_count(&s_looked, looked, x.polls, &s_lost)))) break;
                }
                const uint64_t p_at = p_base + (g + j) % G::kPb * (2 * G::kP) / 16;
                // steps of 16 positions; those behind the sequence are left out, and what is there with them
                const int steps = __shfl_sync(kFull, min(kTile, max(w.s.kv - first - j * kTile, 1) + 15) / 16, 0);
#pragma unroll
                for (int mb = 0; mb < G::kMb; ++mb) {
                    if (!(fine = await_warp(&bars.kv_full[slot], phase, x.polls, &s_lost))) break;
                    tc::fence_after_sync();
                    if (elect_one()) {
                        // d = 64: the second 64 rows of M are the first again (a stride of 0)
                        const uint64_t v_at = tc::desc_mnmajor_sw128(ring_at + slot * G::kSlot, G::kPer == 2 ? kBlock : 0);
                        auto step = [&](int i) {                   // the leading term of P, then the other
                            tc::mma_bf16_ss(tm + G::kO + mb * kRows, v_at + (i & 7) * 2048 / 16, p_at + ((i >> 3) * G::kP + (i & 7) * 2048) / 16,
                                            id_o, j % kFold != 0 || i > 0);
                        };
                        if (steps == kTile / 16) {
#pragma unroll
                            for (int i = 0; i < 2 * kTile / 16; ++i) step(i);
                        } else {
#pragma unroll 1
                            for (int i = 0; i < 2 * kTile / 16; ++i)
                                if ((i & 7) < steps) step(i);
                        }
                        tc::mma_commit(&bars.kv_empty[slot]);
                        if (mb == G::kMb - 1) {
                            tc::mma_commit(&bars.pv_done[(g + j) & 1]);
                            mbar_arrive(&bars.pv_done[(g + j) & 1]);
                        }
                    }
                    __syncwarp();
                    if (++slot == G::kSlots) slot = 0, phase ^= 1;
                }
                if (!fine) break;
            }
            g += n;
            ++items;
        }
    } else {
        // ---------------------------------------------------------------- queries, and values at the ends
        constexpr int kAtOnce = 8;                               // reads of values in flight, 16 bytes each
        constexpr int kQRows = 32 / G::kCpr;                     // rows of Q that the warp asks for at once
        uint32_t items = 0, slot0 = 0, looked = 0;               // slot0: the item's first slot of the ring
        bool fine = true;
        // The next item and its queries, when the last product with the former item's has been made.
        auto next_item = [&]() -> bool {
            do {
                if (!w.next(x)) return false;
            } while (row0 / share >= w.s.rows);
            if (items > 0 && !(fine = await_warp(&bars.q_empty, (items - 1) & 1, x.polls, &s_lost))) return false;
            // rows behind the sequence's last are zeros, whatever q holds there: the votes on the maxima are taken among all
            const int ch = lane % G::kCpr, real = share * w.s.rows - row0;
            int r = lane / G::kCpr, t = (row0 + r) / share, head = row0 + r - t * share;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (((int64_t)w.b * a.T + t) * a.Hq + (int64_t)w.h * share + head) * D + ch * 8;
#pragma unroll 4
            for (; r < rows; r += kQRows) {
                cp_async16(ring_at + kQOff + tile_chunk(kRows, r, ch), q, r < real);
                q += kQRows * D;
                for (head += kQRows; head >= share; head -= share) q += (int64_t)(a.Hq - share) * D;   // the next token's
            }
            cp_async_wait_all();
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.q_full);
            ++items;
            return true;
        };
        bool more = next_item();
        for (int item = 1; more; ++item) {
            const int kv = w.s.kv, n = w.i1 - w.i0, first = w.s.first + w.i0 * kTile;
            const Sight see(a, w.s, row0, row0 + rows, share);
            // Values that are not numbers, at positions that some row does not see, would reach that row
            // as 0 times infinity. They leave a zero in the tile; the rows that do see them get them at
            // the end (`repair` above). The last tile comes after the next item's queries, which it would keep
            // waiting: its scores, the last of this item, are formed by then.
            for (int j = 0; j < n && fine; ++j) {
                if (j == n - 1) more = next_item();
                const int pos = first + j * kTile;
                if (!fine || !see.partial(pos, kTile)) continue;
                if (!(fine = __all_sync(kFull, await_count(&s_ask, ++looked, x.polls, &s_lost)))) break;
                const uint32_t v_slot = slot0 + (j < n - 1 ? 2 * j + 2 : 2 * n - 1) * G::kMb;   // V's first
                // rows 0 .. low - 1 and high .. stop - 1 of the tile; behind them TMA has left zeros, or the product stops
                const int behind = max(kv - pos, 0), stop = min(kTile, min((behind + run - 1) / run * run, (behind + 15) / 16 * 16));
                const int low = min(max(see.lo_max - pos, 0), stop), high = min(max(see.p_min + 1 - pos, low), stop);
                const int ch = lane % G::kCpr, r_lane = lane / G::kCpr;
                unsigned char* const v_at = ring + (v_slot + ch / (8 * G::kPer)) % G::kSlots * G::kSlot;
                for (int r0 = 0; r0 < stop; r0 += kAtOnce * kQRows) {
                    if (r0 >= low && r0 + kAtOnce * kQRows <= high) continue;
                    uint4 y[kAtOnce];
#pragma unroll
                    for (int e = 0; e < kAtOnce; ++e)            // up to 32 rows: all of the tile, if not of the rows before stop
                        y[e] = *reinterpret_cast<const uint4*>(v_at + tile_chunk(kTile, r0 + r_lane + e * kQRows, ch % (8 * G::kPer)));
                    __nv_bfloat162 sum[2] = {__floats2bfloat162_rn(0.f, 0.f), __floats2bfloat162_rn(0.f, 0.f)};
#pragma unroll
                    for (int e = 0; e < kAtOnce; ++e) {
                        sum[0] = taint(y[e].y, taint(y[e].x, sum[0]));
                        sum[1] = taint(y[e].w, taint(y[e].z, sum[1]));
                    }
                    const __nv_bfloat162 both = __hadd2(sum[0], sum[1]);
                    if (__low2float(both) == 0.f && __high2float(both) == 0.f) continue;
#pragma unroll
                    for (int e = 0; e < kAtOnce; ++e) {
                        const int r = r0 + r_lane + e * kQRows;
                        const uint4 z = make_uint4(numbers(y[e].x), numbers(y[e].y), numbers(y[e].z), numbers(y[e].w));
                        if ((r >= low && r < high) || (z.x == y[e].x && z.y == y[e].y && z.z == y[e].z && z.w == y[e].w)) continue;
                        // (behind the sequence, or before what any row sees: nobody's)
                        if (pos + r < kv && pos + r >= see.lo_min) s_not_numbers = item;
                        *reinterpret_cast<uint4*>(v_at + tile_chunk(kTile, r, ch % (8 * G::kPer))) = z;
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) set_count(&s_looked, looked);
            }
            if (!fine) break;
            slot0 += 2 * n * G::kMb;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (s_lost) {
        // Given up: the copies in flight land, and the products end, before the memory goes; and the join is told (a
        // maximum of NaN) that there is no part of this CTA's.
        if (warp >= kSoftWarps && warp < kSoftWarps + kFetch)
            for (uint32_t s = issued > G::kSlots ? issued - G::kSlots : 0; s < issued; ++s)
                if (s % kFetch == warp - kSoftWarps)
                    for (uint32_t i = 0; i < kMaxPolls && !mbar_try_wait(&bars.kv_full[s % G::kSlots], (s / G::kSlots) & 1); ++i) {}
        if (warp == kSoftWarps + kFetch) {
            if (elect_one()) tc::mma_commit(&bars.drain);
            for (uint32_t i = 0; i < kMaxPolls && !mbar_try_wait(&bars.drain, 0); ++i) {}
            __syncwarp();
        }
        if (C > 1)
            for (int i = tid; i < 2 * x.rows; i += G::kThreads) x.parts.m[((size_t)mtile * C + c) * 2 * x.rows + i] = NAN;
    }
    if (warp == kSoftWarps + kFetch) tc::tmem_dealloc(tmem, G::kCols);
    if (tid == 0 && s_lost && a.status_word) atomicOr(a.status_word, kStatusWaitTimeout);
}

template <int D>
cudaError_t launch(const Args& x, const Plan& p, cudaStream_t stream) {
    using G = Cfg<D>;
    static_assert(G::kBytes + 6144 <= 227 * 1024, "shared memory");
    const PagedCache& c = x.a.cache;
    const int run = std::min(kTile, c.page & -c.page);
    CUtensorMap maps[2];
    cudaError_t e = ensure_smem_attr<gdn_paged_attention_tc_kernel<D>>(G::kBytes);
    for (int i = 0; i < 2 && e == cudaSuccess; ++i)
        e = tc::encode_tmap_paged(&maps[i], i ? c.v : c.k, D, x.a.Hk, c.page, c.num_pages, c.head_stride, c.slot_stride,
                                  c.page_stride, run);
    if (e != cudaSuccess) return e;
    Launch l(dim3(p.ctas, p.tiles), G::kThreads, G::kBytes, stream);
    e = cudaLaunchKernelEx(&l.cfg, gdn_paged_attention_tc_kernel<D>, x, maps[0], maps[1], run);
    return e != cudaSuccess ? e : launch_join(x, p, stream);
}
}  // namespace

bool tc_applies(const AttnArgs& a) {
    // TMA copies whole 1024-byte atoms of eight slots, and strides below 2^40 bytes.
    const int64_t most = ((int64_t)1 << 39) - 1;
    if (!a.bf16 || a.cache.page % 8 != 0 || a.cache.page_stride > most || a.cache.slot_stride > most || a.cache.head_stride > most)
        return false;
    const int rows = a.Hq / a.Hk * a.T;
    const double elements = (double)a.B * a.Hk * a.max_pages * a.cache.page * a.d;     // of K that the tables can hold
    if (a.d == 64) return rows > 32 && elements >= 1 << 21;
    if (a.d == 128) return rows > 16 && elements >= 1 << 21;
    return elements >= (rows > 16 ? 1 << 22 : 1 << 23);
}

Plan plan_tc(int sms, int rows) {
    Plan p;
    p.unit = kTile;
    p.extra = kExtra;
    p.tiles = (rows + kRows - 1) / kRows;
    p.rows = p.tiles == 1 ? rows : ((rows + p.tiles - 1) / p.tiles + 15) / 16 * 16;
    p.ctas = std::max(1, sms / p.tiles);
    return p;
}

cudaError_t launch_tc(const Args& x, const Plan& p, cudaStream_t stream) {
    return x.a.d == 64 ? launch<64>(x, p, stream) : x.a.d == 128 ? launch<128>(x, p, stream) : launch<256>(x, p, stream);
}

}  // namespace attn
}  // namespace gdn
