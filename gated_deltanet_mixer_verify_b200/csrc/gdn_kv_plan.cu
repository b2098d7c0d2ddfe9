// gdn_kv_plan.cu -- block tables and slot maps from the requests' lengths, and the pool of cache
// pages behind them: commit of the last block's accept counts, pages returned and handed out,
// one slot per new token (gdn_kv_plan in include/gdn.h).
//
// Whole numbers only: two prefix sums over the sequences (pages returned, pages needed) place
// every sequence's pages on the free list, so the result does not depend on any order of
// execution. One CTA does it, a thread for each sequence, because every step hangs on the sums; it is a chain
// of six dependent reads, bound by their latency: 3 us on the device for one sequence, 7.4 us for 256 of a block of 8
// (11.7 us under a profiler, cold), 8.5 us in all with the slots of 32 prompts of up to 8192. The slots of a block of a few tokens are formed there
// too; those of prompts (one each for tens of thousands of tokens) by a second kernel over all SMs,
// launched as a programmatic dependent.
#include <cuda_runtime.h>

#include <algorithm>

#include "gdn_device.cuh"
#include "gdn_internal.cuh"

namespace gdn {
namespace {

using namespace dev;

constexpr int kMaxThreads = 1024;
constexpr int kMaxWarps = kMaxThreads / 32;
// Up to this many slots one CTA is faster than a second launch.
constexpr int64_t kInlineSlots = 8192;
// A thread copies up to this many pages of its own sequence; more are copied by a warp, the sequences dealt to
// the block's warps in turn (32 prompts of up to 128 pages each: 18.4 us a call by the one warp that their threads are, 10.3 so).
constexpr int kLanePages = 2;

// One sequence's request. want == held where nothing can be done for it.
struct Seq {
    int len, add, held, want, seq_out;
};

__device__ __forceinline__ Seq read_seq(const KvPlanArgs& a, int b, int& status) {
    Seq s;
    const int seq = a.seq_in[b];
    s.held = a.held_in[b];
    int c = a.commit ? a.commit[b] : 0;
    const int block = a.block ? a.block[b] : INT32_MAX;
    int add = a.add ? a.add[b] : a.T;
    c = min(c, block);
    const int64_t room = (int64_t)s.held * a.page;
    if (seq < 0 || s.held < 0 || s.held > a.max_pages || seq > room) {
        status |= kStatusBadLength;
        s.len = 0;
        s.add = 0;
        s.want = s.held;
        s.seq_out = seq;
        return s;
    }
    if (c < 0 || (int64_t)seq + c > room) {
        status |= kStatusBadAccept;
        c = 0;
    }
    if (add < -1 || add > a.T) {
        status |= kStatusBadLength;
        add = 0;
    }
    s.len = add < 0 ? 0 : seq + c;
    s.add = add < 0 ? 0 : add;
    s.seq_out = s.len;
    // len + add <= 2^30 + 2^20
    s.want = (int)(((unsigned)(s.len + s.add) + (unsigned)a.page - 1) / (unsigned)a.page);
    if (s.want > a.max_pages) {
        status |= kStatusNoPages;
        s.want = s.held;
        s.add = 0;
    }
    return s;
}

// Inclusive sum over the block's threads; *total receives the whole sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* part, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();   // part may still be read from the scan before
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int64_t p = lane < warps ? part[lane] : 0;         // every warp sums the warps' totals
    int64_t incl = p;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += y;
    }
    *total = __shfl_sync(kFull, incl, 31);
    return x + __shfl_sync(kFull, incl - p, warp);
}

// A warp's copy of n entries, eight reads in flight: to(i, from(i)).
template <typename From, typename To>
__device__ __forceinline__ void warp_copy(int n, int lane, From from, To to) {
    for (int i = lane; i < n; i += 256) {
        int v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + 32 * k < n) v[k] = from(i + 32 * k);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + 32 * k < n) to(i + 32 * k, v[k]);
    }
}

__global__ void __launch_bounds__(kMaxThreads) gdn_kv_plan_kernel(const __grid_constant__ KvPlanArgs a, bool slots_here) {
    __shared__ int64_t part[kMaxWarps];
    __shared__ unsigned long long s_granted;
    __shared__ int s_len[kMaxThreads], s_q[kMaxThreads], s_held[kMaxThreads], s_k0[kMaxThreads], s_n[kMaxThreads];
    // the slot kernel may take its place on the SMs now; it waits for this one to end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const int tiles = (a.B + nt - 1) / nt;
    int status = 0;
    int count = *a.count_in;
    Seq s = {};
    if (tid < a.B) s = read_seq(a, tid, status);
    if (count < 0 || count > a.num_pages) {
        if (tid == 0) status |= kStatusBadLength;
        count = min(max(count, 0), a.num_pages);
    }
    if (tid == 0) s_granted = 0;

    // Returned pages onto the free list, in order of b and of the pages within b.
    int64_t carry = count;
    for (int tile = 0; tile < tiles; ++tile) {
        const int b = tile * nt + tid;
        if (tile > 0) {
            s = Seq{};
            if (b < a.B) s = read_seq(a, b, status);
        }
        const int back = max(s.held - s.want, 0);
        int64_t total;
        const int64_t at = carry + block_scan(back, part, &total) - back;
        const int to = (int)min(at, (int64_t)a.num_pages), n = min(back, a.num_pages - to);
        if (n <= kLanePages)
            for (int i = 0; i < n; ++i) a.free_list[to + i] = a.table[(size_t)b * a.max_pages + s.want + i];
        // (in these loops the arrays are the next tile's again behind its scan's barriers)
        s_n[tid] = n;
        s_k0[tid] = to;
        s_held[tid] = s.want;
        if (__syncthreads_or(n > kLanePages))
            for (int j = warp; j < min(nt, a.B - tile * nt); j += nt / 32) {
                if (s_n[j] <= kLanePages) continue;
                const int32_t* from = a.table + (size_t)(tile * nt + j) * a.max_pages + s_held[j];
                int32_t* onto = a.free_list + s_k0[j];
                warp_copy(s_n[j], lane, [&](int i) { return from[i]; }, [&](int i, int v) { onto[i] = v; });
            }
        carry += total;
    }
    const int64_t have = carry < a.num_pages ? carry : a.num_pages;
    if (carry > a.num_pages) status |= kStatusBadLength;   // some page was free, or somebody else's, already
    __syncthreads();

    // Pages handed out from the top, in the same order, while they last; then the slots.
    carry = 0;
    for (int tile = 0; tile < tiles; ++tile) {
        const int b0 = tile * nt, b = b0 + tid;
        if (tiles > 1) {
            s = Seq{};
            int seen = 0;
            if (b < a.B) s = read_seq(a, b, seen);
        }
        const int need = max(s.want - s.held, 0);
        int64_t total;
        const int64_t upto = carry + block_scan(need, part, &total);
        carry += total;
        const bool granted = need == 0 || upto <= have;
        if (!granted) status |= kStatusNoPages;
        const int k0 = granted ? (int)(upto - need) : 0;
        const int now = granted ? s.want : s.held, q = granted ? s.add : 0;
        s_len[tid] = s.len;
        s_q[tid] = q;
        s_held[tid] = s.held;
        s_k0[tid] = k0;
        if (need > 0 && granted) atomicMax(&s_granted, (unsigned long long)upto);
        const int take = granted ? need : 0;
        if (take <= kLanePages)
            for (int i = 0; i < take; ++i) a.table[(size_t)b * a.max_pages + s.held + i] = a.free_list[have - 1 - k0 - i];
        s_n[tid] = take;
        // every thread has read this tile's counts: they may be written in place
        if (__syncthreads_or(take > kLanePages))
            for (int j = warp; j < min(nt, a.B - b0); j += nt / 32) {
                if (s_n[j] <= kLanePages) continue;
                const int32_t* top = a.free_list + (have - 1 - s_k0[j]);
                int32_t* row = a.table + (size_t)(b0 + j) * a.max_pages + s_held[j];
                warp_copy(s_n[j], lane, [&](int i) { return top[-i]; }, [&](int i, int v) { row[i] = v; });
            }
        if (b < a.B) {
            a.seq_out[b] = s.seq_out;
            a.held_out[b] = now;
            a.kv_len[b] = s.len + q;
            a.q_len[b] = q;
        }
        if (slots_here) {
            // A new page's id is read from the free list itself, so a slot waits for no table write.
            const unsigned n = (unsigned)min(nt, a.B - b0) * (unsigned)a.T, T = (unsigned)a.T, page = (unsigned)a.page;
            int64_t* slots = a.slots + (size_t)b0 * T;
            for (unsigned i0 = tid; i0 < n; i0 += 4 * nt) {
                int64_t slot[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const unsigned i = i0 + k * nt, j = i / T, t = i - j * T;
                    slot[k] = -1;
                    if (i < n && (int)t < s_q[j]) {
                        const unsigned pos = (unsigned)s_len[j] + t, pg = pos / page;
                        const int id = (int)pg < s_held[j] ? a.table[(size_t)(b0 + j) * a.max_pages + pg]
                                                           : a.free_list[have - 1 - s_k0[j] - ((int)pg - s_held[j])];
                        if ((unsigned)id < (unsigned)a.num_pages) slot[k] = (int64_t)id * page + (pos - pg * page);
                        else status |= kStatusBadPage;
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i0 + k * nt < n) slots[i0 + k * nt] = slot[k];
            }
        }
        if (tile + 1 < tiles) __syncthreads();      // s_len and the others are the next tile's
    }
    if (tid == 0) *a.count_out = (int)(have - (int64_t)s_granted);
    if (a.status_word) {
        status = __reduce_or_sync(kFull, status);
        if (lane == 0 && status) atomicOr(a.status_word, status);
    }
}

// The slots of B T rows from the counts and tables that the kernel above left.
__global__ void __launch_bounds__(256) gdn_kv_slots_kernel(const __grid_constant__ KvPlanArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const unsigned T = (unsigned)a.T, page = (unsigned)a.page;
    const int64_t n = (int64_t)a.B * T;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int b = n >> 32 ? (int)(i / T) : (int)((uint32_t)i / T);
        const int t = (int)(i - (int64_t)b * T), q = a.q_len[b];
        int64_t slot = -1;
        if (t < q) {
            const unsigned pos = (unsigned)(a.kv_len[b] - q + t), pg = pos / page;
            const int id = a.table[(size_t)b * a.max_pages + pg];
            if ((unsigned)id < (unsigned)a.num_pages) slot = (int64_t)id * page + (pos - pg * page);
            else if (a.status_word) atomicOr(a.status_word, kStatusBadPage);
        }
        a.slots[i] = slot;
    }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
    const int64_t slots = (int64_t)a.B * a.T;
    const bool here = slots <= kInlineSlots;
    const int64_t busy = std::max<int64_t>(a.B, here ? slots : 0);
    // prompts: every warp has pages to copy
    const int threads = !here ? kMaxThreads : (int)std::min<int64_t>(kMaxThreads, std::max<int64_t>(64, (busy + 31) / 32 * 32));
    gdn_kv_plan_kernel<<<1, threads, 0, stream>>>(a, here);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || here) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((slots + 255) / 256, 148 * 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_kv_slots_kernel, a);
}

}  // namespace gdn
