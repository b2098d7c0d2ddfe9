// gdn_attn.cu -- attention of one new token or a verify block over the paged cache
// (gdn_paged_attention in include/gdn.h): the streaming kernel, and the choice of kernel.
//
// For few rows the cache is read once and each value meets a handful of queries: the kernel is a
// stream from HBM. Every warp is a unit of its own: it fetches 16 positions at a time (keys and
// values of one key head) into a ring in shared memory with 16-byte asynchronous copies, finding
// each position's page itself, so pages of any size and any strides stream alike, and works on them
// with warp matrix instructions while the next ones arrive. No barrier stands in the loop. The
// rows of a key head (block rows x heads that share it) are the 16 rows of the matrix products:
//   s = q k^T (base-2 exponents), running maximum m and sum l per row, o = o 2^(m - m') + 2^(s - m') v.
// A warp's maxima, totals and sums are joined with the other warps' when the CTA leaves the item.
//
// Bound: HBM. Measured, bf16, one row per sequence: 64 sequences of 500 .. 16,384 positions, 32 heads over 8, d 128
// (2.2 GB) 356 to 403 us a call by the machine, 84 to 95% of the measured copy rate; 128 sequences of 1 .. 2048, 16 heads
// over 16 (1.07 GB) 204 to 218 us, 75 to 80% (2,048 short items: their beginnings and ends); one sequence of 1,024 12.7 us, latency: the page
// numbers, the values and the join one after another. fp32 (three products for one, 16 sequences, window 1000) 21 us, latency too.
// One wave of CTAs, because more cost: one, two, three, four waves 352, 354, 361, 367 and 193, 197, 203, 209 us (in a graph, before
// the last steps on precision). An item counts as three units more: with 2, 3, 5, 7 the second case took 208, 193, 188, 193 us then,
// all others the same within 2% but 32 sequences of 100 .. 2048 (d 128) 27.0, 26.1, 26.7, 28.1.
//
// Precision. bf16 products are exact in fp32. The weights 2^(s - m) enter the second product as two
// bf16 terms (2^-17 relative), because one (2^-9) would be as large as the rounding of a bf16
// result; the matrix units have the room. fp32 operands are split into two tf32 terms each, and the
// three products that matter are added (2^-22). Statistics and sums are fp32. The matrix units cut where they
// add, always towards zero, so a long fp32 sum formed in them drifts by 2^-24 with every step: there
// they form short sums only, and ordinary additions, which round, put those together.
// Measured, 64 sequences of 4096 positions, 16 heads over 4, values of one, mean error of the outputs (formed in the units:
// all in them): d 64 -5.9e-8 (-1.4e-6), 136 us (133); d 128 -6.5e-8 (-1.8e-6), 371 us (342); d 256 -5.8e-8
// (-2.5e-6), 956 us (821); summing each half of a stage apart -4e-8, 137, 393, 1064 us. (With the look at scores that are
// NaN they take 139, 387 and 979.) bf16, 80 sequences of 16,384: d 64
// -2.9e-8 (-2.4e-6), d 128 -3.3e-8 (-3.0e-6); the first and second case above take 2 and 4% longer for it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_attn.cuh"
#include "gdn_attn_tc.cuh"

namespace gdn {
namespace attn {
namespace {

using namespace dev;

// Geometry of the streaming kernel. A stage is 16 positions of keys and values.
template <typename E, int D>
struct Geo {
    static constexpr int kRow = D * (int)sizeof(E);              // bytes of one position
    static constexpr int kStage = 2 * 16 * kRow;
    static constexpr int kWarps = kStage <= 16384 ? 4 : 3;
    static constexpr int kStages = kStage <= 4096 ? 4 : kStage <= 16384 ? 3 : 2;
    static constexpr int kCtasPerSm = kStage <= 4096 ? 3 : kStage <= 8192 ? 2 : 1;
    static constexpr int kUnit = 16 * kWarps;                    // positions per unit
    static constexpr int kExtra = 3;                             // units that an item costs besides
    static constexpr int kMaxTiles = D <= 128 ? 2 : 1;           // 16-row tiles a warp's registers hold
    static constexpr int kRing = kStages * kStage;               // bytes per warp
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    // a source size of 0 fills the 16 bytes with zeros and reads nothing
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo exactly, hi rounded to the 11 bits of tf32 (half away from zero), lo (12 bits at most) left to
// the matrix unit, which drops what is below its 11 bits: 2^-23 of x. Cutting instead of rounding would lose
// four times that, always towards zero.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 g = __floats2bfloat162_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&g);
}

// Where 16-byte chunk `chunk` of row `row` lies: the rows of a tile are permuted within themselves so
// that the eight rows (bf16: one 16-byte chunk of each; fp32: two chunks of four) that a matrix
// fragment reads at once lie in different banks.
template <typename E>
__device__ __forceinline__ int swizzle(int row, int chunk) {
    if constexpr (sizeof(E) == 2) return chunk ^ (row & 7);
    else return chunk ^ (((row ^ (row >> 2)) & 3) << 1);
}
template <typename E, int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int row, int chunk) {
    return base + row * (D * (int)sizeof(E)) + swizzle<E>(row, chunk) * 16;
}
__device__ __forceinline__ float lds(uint32_t addr) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ float2 lds2(uint32_t addr) {
    float2 x;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(addr) : "memory");
    return x;
}
// Element (row, col) of a tile as fp32.
template <typename E, int D>
__device__ __forceinline__ float element(const unsigned char* tile, int row, int col) {
    constexpr int per = 16 / sizeof(E);
    const unsigned char* p = tile + row * (D * (int)sizeof(E)) + swizzle<E>(row, col / per) * 16 + col % per * (int)sizeof(E);
    return to_f(*reinterpret_cast<const E*>(p));
}

template <typename E, int D>
__device__ __forceinline__ void set_zero(unsigned char* tile, int row, int col) {
    constexpr int per = 16 / sizeof(E);
    unsigned char* p = tile + row * (D * (int)sizeof(E)) + swizzle<E>(row, col / per) * 16 + col % per * (int)sizeof(E);
    *reinterpret_cast<E*>(p) = E(0.f);
}

// s[j] += q k^T for the 16 positions of a stage (j: its two halves), one 16-row tile of q.
template <int D>
__device__ __forceinline__ void scores(const __nv_bfloat16*, uint32_t q, uint32_t k, int lane, float (&s)[2][4]) {
    const int row = lane & 15, half = lane >> 4;
    const int krow = (lane & 7) + (lane >> 4) * 8, khalf = (lane >> 3) & 1;
    float t[2][4] = {};   // odd steps: two chains of products instead of one
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t a[4], b[4];
        ldmatrix4(chunk_at<__nv_bfloat16, D>(q, row, 2 * i + half), a);
        ldmatrix4(chunk_at<__nv_bfloat16, D>(k, krow, 2 * i + khalf), b);
        float(&d)[2][4] = (i & 1) ? t : s;
        mma_bf16(d[0], a, b[0], b[1]);
        mma_bf16(d[1], a, b[2], b[3]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] += t[j][e];
}
template <int D>
__device__ __forceinline__ void scores(const float*, uint32_t q, uint32_t k, int lane, float (&s)[2][4]) {
    // column pairs 2 (lane % 4), + 1 of each step serve as the step's k index lane % 4 and + 4, in
    // q and k alike
    const int row = lane >> 2, pair = lane & 3;
    float t[2][4] = {}, u[2][4] = {};
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        const int chunk = 2 * i + (pair >> 1), in = (pair & 1) * 8;
        const float2 q0 = lds2(chunk_at<float, D>(q, row, chunk) + in), q1 = lds2(chunk_at<float, D>(q, row + 8, chunk) + in);
        uint32_t ah[4], al[4];
        split_tf32(q0.x, ah[0], al[0]);
        split_tf32(q1.x, ah[1], al[1]);
        split_tf32(q0.y, ah[2], al[2]);
        split_tf32(q1.y, ah[3], al[3]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 kk = lds2(chunk_at<float, D>(k, row + 8 * j, chunk) + in);
            uint32_t bh[2], bl[2];
            split_tf32(kk.x, bh[0], bl[0]);
            split_tf32(kk.y, bh[1], bl[1]);
            mma_tf32(t[j], al, bh[0], bh[1]);
            mma_tf32(t[j], ah, bl[0], bl[1]);
            mma_tf32(u[j], ah, bh[0], bh[1]);
        }
        if (i % 4 == 3)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[j][e] += u[j][e];
                    u[j][e] = 0.f;
                }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] += t[j][e];
}

// o += p v for the 16 positions of a stage, MT row tiles (a value fragment serves all of them).
template <int D, int MT>
__device__ __forceinline__ void products(const __nv_bfloat16*, const float (&p)[MT][2][4], uint32_t v, int lane,
                                         float (&o)[MT][D / 8][4]) {
    uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            split_bf16(p[m][j][0], p[m][j][1], hi[m][2 * j], lo[m][2 * j]);
            split_bf16(p[m][j][2], p[m][j][3], hi[m][2 * j + 1], lo[m][2 * j + 1]);
        }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t b[4];
        ldmatrix4_trans(chunk_at<__nv_bfloat16, D>(v, lane & 15, 2 * i + (lane >> 4)), b);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float t[2][4] = {};                                  // the stage's sum, formed apart
            mma_bf16(t[0], hi[m], b[0], b[1]);
            mma_bf16(t[1], hi[m], b[2], b[3]);
            mma_bf16(t[0], lo[m], b[0], b[1]);
            mma_bf16(t[1], lo[m], b[2], b[3]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[m][2 * i + j][e] += t[j][e];
        }
    }
}
template <int D, int MT>
__device__ __forceinline__ void products(const float*, const float (&p)[MT][2][4], uint32_t v, int lane,
                                         float (&o)[MT][D / 8][4]) {
    // position pairs 2 (lane % 4), + 1 of each half serve as its k index lane % 4 and + 4
    const int col = lane >> 2, pair = lane & 3;
    uint32_t ph[MT][2][4], pl[MT][2][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            split_tf32(p[m][j][0], ph[m][j][0], pl[m][j][0]);
            split_tf32(p[m][j][2], ph[m][j][1], pl[m][j][1]);
            split_tf32(p[m][j][1], ph[m][j][2], pl[m][j][2]);
            split_tf32(p[m][j][3], ph[m][j][3], pl[m][j][3]);
        }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const int chunk = 2 * i + (col >> 2), in = (col & 3) * 4;
        float t[MT][4] = {};                                     // the stage's sum, formed apart
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 8 * j + 2 * pair;
            uint32_t bh[2], bl[2];
            split_tf32(lds(chunk_at<float, D>(v, row, chunk) + in), bh[0], bl[0]);
            split_tf32(lds(chunk_at<float, D>(v, row + 1, chunk) + in), bh[1], bl[1]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                mma_tf32(t[m], pl[m][j], bh[0], bh[1]);
                mma_tf32(t[m], ph[m][j], bl[0], bl[1]);
                mma_tf32(t[m], ph[m][j], bh[0], bh[1]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[m][i][e] += t[m][e];
    }
}

// q k of row `row` and position `pos` of a stage, for a score whose tf32 terms gave NaN: one of an infinity is the
// infinity less itself. In plain fp32 it is what the formula gives, an infinity or a number among it.
template <int D>
__device__ __noinline__ float plain_score(const unsigned char* q, const unsigned char* k, int row, int pos) {
    float s = 0.f;
    for (int i = 0; i < D; ++i) s = fmaf(element<float, D>(q, row, i), element<float, D>(k, pos, i), s);
    return s;
}

// For a stage whose values are not all numbers while some row does not see all of its positions: 0
// times infinity would reach that row in the product. So what is not a number goes straight to
// the sums of the rows that see it, and leaves a zero in the stage; the product that follows is the
// one the other rows would have had without it, bit for bit.
template <typename E, int D, int MT>
__device__ __forceinline__ void take_out_non_numbers(unsigned char* v, const uint32_t (&seen)[MT][2], int lane,
                                                     float (&o)[MT][D / 8][4]) {
#pragma unroll 1
    for (int key = 0; key < 16; ++key)
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = element<E, D>(v, key, 8 * i + 2 * (lane & 3) + e);
                if (is_number<E>(x)) continue;
                x = as_infinite(x);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (seen[m][0] >> key & 1) o[m][i][e] += x;
                    if (seen[m][1] >> key & 1) o[m][i][2 + e] += x;
                }
            }
    __syncwarp();
    for (int i = lane; i < 16 * D; i += 32)
        if (!is_number<E>(element<E, D>(v, i / D, i % D))) set_zero<E, D>(v, i / D, i % D);
    __syncwarp();
}

// grid (C, row tiles). Shared memory: the warps' rings, then the CTA's 16 MT query rows.
template <typename E, int D, int MT>
__global__ void __launch_bounds__(Geo<E, D>::kWarps * 32, Geo<E, D>::kCtasPerSm)
gdn_paged_attention_kernel(const __grid_constant__ Args x) {
    using G = Geo<E, D>;
    constexpr int NW = G::kWarps, NT = NW * 32, S = G::kStages;
    constexpr int CPR = G::kRow / 16;                  // 16-byte chunks per position
    constexpr int LOADS = 16 * CPR / 32;               // per lane, of keys and of values
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t s_start[NW + 2];
    __shared__ float s_m[NW][16 * MT], s_l[NW][16 * MT];
    const AttnArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = gridDim.x, c = blockIdx.x, tile = blockIdx.y;
    // The join kernel may take its place on the SMs from here on; it waits for this one to end.
    grid_wait();
    grid_release();
    int kv0, rows0;
    ask_counts(a, kv0, rows0);
    const Start at = find_start<NT, G::kUnit, G::kExtra>(x, s_start, c, C, tile, kv0, rows0);

    unsigned char* ring = smem + warp * G::kRing;
    unsigned char* q_tile = smem + NW * G::kRing;
    const uint32_t ring_at = smem_u32(ring), q_at = smem_u32(q_tile);
    const int share = a.Hq / a.Hk, row0 = tile * x.rows, all_rows = share * a.T;
    const uint32_t page = (uint32_t)a.cache.page;
    const E* kc = static_cast<const E*>(a.cache.k);
    const E* vc = static_cast<const E*>(a.cache.v);

    Walk<G::kUnit, G::kExtra> w(at);
    while (w.next(x)) {
        if (row0 / share >= w.s.rows) continue;                                // none of this tile's rows
        const Seq& s = w.s;
        const int b = w.b, h = w.h, i0 = w.i0, i1 = w.i1;

        // the item's query rows; zeros for rows behind the sequence's last, whatever q holds there
        for (int i = tid; i < 16 * MT * CPR; i += NT) {
            const int r = i / CPR, ch = i - r * CPR, row = row0 + r;
            uint4 z = make_uint4(0, 0, 0, 0);
            if (row < share * s.rows) {
                const int t = row / share;
                const int64_t qr = ((int64_t)b * a.T + t) * a.Hq + (int64_t)h * share + (row - t * share);
                z = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) + qr * G::kRow + ch * 16);
            }
            *reinterpret_cast<uint4*>(q_tile + r * G::kRow + swizzle<E>(r, ch) * 16) = z;
        }
        __syncthreads();

        const Sight see(a, s, row0, min(row0 + 16 * MT, all_rows), share);
        const int p0 = see.p0, p_min = see.p_min, lo_min = see.lo_min, lo_max = see.lo_max;

        // this warp's stages: 16 positions from 16 g on, g = g_first, + NW, ... below g_end
        const int first = s.first + i0 * G::kUnit;
        const int g_end = min((s.first + i1 * G::kUnit) / 16, (s.kv + 15) / 16);
        int g_load = first / 16 + warp, g = g_load;

        // Lanes 0 .. 15 each look one position up: its page, its offset in the cache (-1: not there).
        int id = -1;
        auto look_up = [&](int gg) {
            const int pos = gg * 16 + lane;
            id = -1;
            if (lane < 16 && gg < g_end && pos < s.kv && pos >= lo_min) {
                id = a.table[(int64_t)b * a.max_pages + (uint32_t)pos / page];
                if ((unsigned)id >= (unsigned)a.cache.num_pages) {
                    if (a.status_word) atomicOr(a.status_word, kStatusBadPage);
                    id = -1;
                }
            }
        };
        uint32_t there[S];           // the stage's positions that are there, one bit each
        auto fetch = [&](int stage) -> uint32_t {
            const uint32_t in_page = (uint32_t)(g_load * 16 + (lane & 15)) % page;
            const int64_t off = id * a.cache.page_stride + (int64_t)in_page * a.cache.slot_stride + h * a.cache.head_stride;
            const uint32_t mask = __ballot_sync(kFull, id >= 0);
            const uint32_t k_at = ring_at + stage * G::kStage, v_at = k_at + G::kStage / 2;
            if (g_load < g_end) {
#pragma unroll
                for (int i = 0; i < LOADS; ++i) {
                    const int n = i * 32 + lane, row = n / CPR, ch = n - row * CPR;
                    const int64_t o = __shfl_sync(kFull, off, row);
                    const bool take = mask >> row & 1;
                    const int64_t e = take ? o + ch * (16 / (int)sizeof(E)) : 0;
                    cp_async16(chunk_at<E, D>(k_at, row, ch), kc + e, take);
                    cp_async16(chunk_at<E, D>(v_at, row, ch), vc + e, take);
                }
            }
            cp_async_commit();
            g_load += NW;
            look_up(g_load);
            return mask;
        };

        float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
            m[i][0] = m[i][1] = -INFINITY;
            l[i][0] = l[i][1] = 0.f;
        }

        look_up(g_load);
#pragma unroll
        for (int i = 0; i < S - 1; ++i) there[i] = fetch(i);
        while (g < g_end) {
#pragma unroll
            for (int stage = 0; stage < S; ++stage) {      // unrolled so that `there` stays in registers
                if (g >= g_end) break;
                there[(stage + S - 1) % S] = fetch((stage + S - 1) % S);
                cp_async_wait<S - 1>();
                __syncwarp();
                const uint32_t k_at = ring_at + stage * G::kStage, v_at = k_at + G::kStage / 2;
                const uint32_t mask = there[stage];
                const bool all = mask == 0xffffu && g * 16 + 15 <= p_min && g * 16 >= lo_max;
                float p[MT][2][4];
                uint32_t seen[MT][2];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[i][j][e] = 0.f;
                    scores<D>(static_cast<const E*>(nullptr), q_at + i * 16 * G::kRow, k_at, lane, p[i]);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[i][j][e] *= x.c;
                    if (!all) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            // bits of the positions that this row sees
                            const int row = row0 + 16 * i + (lane >> 2) + 8 * r;
                            const int pr = p0 + row / share;
                            const int hi = pr - g * 16, lo = a.window > 0 ? pr - a.window + 1 - g * 16 : 0;
                            uint32_t bits = hi < 0 ? 0u : hi >= 15 ? 0xffffu : (2u << hi) - 1u;
                            if (lo > 0) bits = lo >= 16 ? 0u : bits & (0xffffu << lo);
                            bits &= mask;
                            seen[i][r] = bits;
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!(bits >> (8 * j + 2 * (lane & 3) + e) & 1)) p[i][j][2 * r + e] = -INFINITY;
                        }
                    }
                    if constexpr (sizeof(E) == 4) {
                        // (what is not seen is -infinity by now)
                        if (isnan(((p[i][0][0] + p[i][0][1]) + (p[i][0][2] + p[i][0][3])) + ((p[i][1][0] + p[i][1][1]) + (p[i][1][2] + p[i][1][3])))) {
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (isnan(p[i][j][e]))
                                        p[i][j][e] = x.c * plain_score<D>(q_tile, ring + stage * G::kStage, 16 * i + (lane >> 2) + 4 * (e & 2),
                                                                          8 * j + 2 * (lane & 3) + (e & 1));
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float top = fmaxf(fmaxf(p[i][0][2 * r], p[i][0][2 * r + 1]), fmaxf(p[i][1][2 * r], p[i][1][2 * r + 1]));
                        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                        if (top > m[i][r]) {
                            const float k = exp2_approx(m[i][r] - top);     // 0 the first time
                            m[i][r] = top;
                            l[i][r] *= k;
#pragma unroll
                            for (int j = 0; j < D / 8; ++j) {
                                o[i][j][2 * r] *= k;
                                o[i][j][2 * r + 1] *= k;
                            }
                        }
                        const float use = m[i][r] == -INFINITY ? 0.f : m[i][r];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                p[i][j][2 * r + e] = exp2_approx(p[i][j][2 * r + e] - use);
                                l[i][r] += p[i][j][2 * r + e];
                            }
                    }
                }
                if (!all) {
                    unsigned char* v = ring + stage * G::kStage + G::kStage / 2;
                    bool numbers = true;
                    for (int i = lane; i < 16 * D; i += 32) numbers &= is_number<E>(element<E, D>(v, i / D, i % D));
                    if (!__all_sync(kFull, numbers)) take_out_non_numbers<E, D, MT>(v, seen, lane, o);
                }
                products<D, MT>(static_cast<const E*>(nullptr), p, v_at, lane, o);
                g += NW;
                __syncwarp();      // the stage is overwritten by the next fetch
            }
        }
        cp_async_wait<0>();
        __syncwarp();

        // The warps' results, joined through their rings.
        float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[i][r] += __shfl_xor_sync(kFull, l[i][r], 1);
                l[i][r] += __shfl_xor_sync(kFull, l[i][r], 2);
                const int row = 16 * i + (lane >> 2) + 8 * r;
                if ((lane & 3) == 0) {
                    s_m[warp][row] = m[i][r];
                    s_l[warp][row] = l[i][r];
                }
#pragma unroll
                for (int j = 0; j < D / 8; ++j)
                    *reinterpret_cast<float2*>(mine + row * D + 8 * j + 2 * (lane & 3)) = make_float2(o[i][j][2 * r], o[i][j][2 * r + 1]);
            }
        }
        __syncthreads();
        const size_t part = (((size_t)tile * C + c) * 2 + w.slot) * x.rows;
        for (int i = tid; i < 16 * MT * (D / 4); i += NT) {
            const int r = i / (D / 4), col = (i - r * (D / 4)) * 4, row = row0 + r, t = row / share;
            if (row >= all_rows || t >= s.rows) continue;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < NW; ++j) top = fmaxf(top, s_m[j][r]);
            const float use = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                const float k = exp2_approx(s_m[j][r] - use);
                sum = fmaf(k, s_l[j][r], sum);
                fma4(y, k, *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + j * G::kRing) + r * D + col));
            }
            if (isnan((y.x + y.y) + (y.z + y.w)) && !isnan(sum)) {
                const int pr = p0 + t, from = max(first, a.window > 0 ? pr - a.window + 1 : 0), to = min(min(s.kv, pr + 1), s.first + i1 * G::kUnit);
                float* const e[4] = {&y.x, &y.y, &y.z, &y.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!isnan(*e[j])) continue;
                    const float z = sum_non_numbers<E>(a, b, h, col + j, from, to);
                    if (z != 0.f) *e[j] = z;
                }
            }
            if (w.whole) {
                const float inv = 1.f / sum;
                if (sum == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
                const int64_t out = ((int64_t)b * a.T + t) * a.Hq + (int64_t)h * share + (row - t * share);
                store_o4(a, out * D + col, sum == 0.f ? y : make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
                if (col == 0 && a.lse) a.lse[out] = (use + log2f(sum)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(x.parts.o + (part + r) * D + col) = y;
                if (col == 0) {
                    x.parts.m[part + r] = top;
                    x.parts.l[part + r] = sum;
                }
            }
        }
        __syncthreads();   // the rings and the queries are the next item's
    }
}

// Row tiles a warp takes at once: as many as hold the rows, at most what its registers hold.
template <typename E, int D>
Plan plan_stream(int sms, int rows) {
    using G = Geo<E, D>;
    int mt = 1;
    while (mt < G::kMaxTiles && 16 * mt < rows) mt *= 2;
    Plan p;
    p.unit = G::kUnit;
    p.extra = G::kExtra;
    p.rows = 16 * mt;
    p.tiles = (rows + p.rows - 1) / p.rows;
    p.ctas = std::max(1, sms * G::kCtasPerSm / p.tiles);
    return p;
}

template <typename E, int D, int MT>
cudaError_t launch_stream(const Args& x, const Plan& p, cudaStream_t stream) {
    using G = Geo<E, D>;
    constexpr int bytes = G::kWarps * G::kRing + 16 * MT * G::kRow;
    cudaError_t e = ensure_smem_attr<gdn_paged_attention_kernel<E, D, MT>>(bytes);
    if (e != cudaSuccess) return e;
    Launch l(dim3(p.ctas, p.tiles), G::kWarps * 32, bytes, stream);
    e = cudaLaunchKernelEx(&l.cfg, gdn_paged_attention_kernel<E, D, MT>, x);
    return e != cudaSuccess ? e : launch_join(x, p, stream);
}

template <typename E, int D>
cudaError_t launch_rows(const Args& x, const Plan& p, cudaStream_t stream) {
    if (p.rows == 16) return launch_stream<E, D, 1>(x, p, stream);
    if constexpr (D <= 128)
        if (p.rows == 32) return launch_stream<E, D, 2>(x, p, stream);
    return cudaErrorInvalidValue;
}

Plan plan_of(int sms, int rows, int d, bool bf16) {
    if (bf16)
        return d == 64 ? plan_stream<__nv_bfloat16, 64>(sms, rows)
                       : d == 128 ? plan_stream<__nv_bfloat16, 128>(sms, rows) : plan_stream<__nv_bfloat16, 256>(sms, rows);
    return d == 64 ? plan_stream<float, 64>(sms, rows)
                   : d == 128 ? plan_stream<float, 128>(sms, rows) : plan_stream<float, 256>(sms, rows);
}

}  // namespace
}  // namespace attn

size_t paged_attention_workspace_bytes(int B, int T, int Hq, int Hk, int d, bool bf16) {
    using namespace attn;
    if (B == 0) return 0;
    const int rows = Hq / Hk * T;
    size_t n = parts_bytes(plan_of(kMaxSms, rows, d, bf16), d);
    if (bf16) n = std::max(n, parts_bytes(plan_tc(kMaxSms, rows), d));
    return n;
}

cudaError_t launch_paged_attention(const AttnArgs& a, cudaStream_t stream) {
    using namespace attn;
    int sms = 0;
    cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return e;
    sms = std::min(sms, kMaxSms);
    const bool on_tc = tc_applies(a);
    const int rows = a.Hq / a.Hk * a.T;
    const Plan p = on_tc ? plan_tc(sms, rows) : plan_of(sms, rows, a.d, a.bf16);
    Args x;
    x.a = a;
    x.parts = parts_at(a.workspace, p, a.d);
    x.rows = p.rows;
    x.c = a.scale * kLog2e;
    x.polls = a.polls ? a.polls : kMaxPolls;
    if (on_tc) return launch_tc(x, p, stream);
    if (a.bf16)
        return a.d == 64 ? launch_rows<__nv_bfloat16, 64>(x, p, stream)
                         : a.d == 128 ? launch_rows<__nv_bfloat16, 128>(x, p, stream) : launch_rows<__nv_bfloat16, 256>(x, p, stream);
    return a.d == 64 ? launch_rows<float, 64>(x, p, stream)
                     : a.d == 128 ? launch_rows<float, 128>(x, p, stream) : launch_rows<float, 256>(x, p, stream);
}

}  // namespace gdn
