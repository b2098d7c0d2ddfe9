// gdn_kv_plan.cu -- block tables and slot maps from the requests' lengths, and the pool of cache
// pages behind them: commit of the last block's accept counts, pages returned and handed out,
// one slot per new token (gdn_kv_plan in include/gdn.h).
//
// Whole numbers only: two prefix sums over the sequences (pages returned, pages needed) place
// every sequence's pages on the free list, so the result does not depend on any order of
// execution. One launch: a single CTA, or one cluster whose CTAs all compute the same sums and
// share the copies and the slots.
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.cuh"

namespace gdn {
namespace {

using namespace dev;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
// Above this many slots one SM's stores and divisions outweigh a cluster's launch and barriers.
constexpr int64_t kOneCtaSlots = 16384;
// A lane copies up to this many pages of its own sequence; more are copied by the whole warp.
constexpr int kLanePages = 2;

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster; orders their global-memory accesses as well.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One sequence's request. want == held where nothing can be done for it.
struct Seq {
    int len, add, held, want, seq_out;
    bool stuck;   // its own counts cannot be, or it would not fit its block table: nothing is added
};

__device__ __forceinline__ Seq read_seq(const KvPlanArgs& a, int b, int& status) {
    Seq s;
    const int seq = a.seq_in[b];
    s.held = a.held_in[b];
    int c = a.commit ? a.commit[b] : 0;
    if (a.block) c = min(c, a.block[b]);
    int add = a.add ? a.add[b] : a.T;
    const int64_t room = (int64_t)s.held * a.page;
    s.stuck = false;
    if (seq < 0 || s.held < 0 || s.held > a.max_pages || seq > room) {
        status |= kStatusBadLength;
        s.len = 0;
        s.add = 0;
        s.want = s.held;
        s.seq_out = seq;
        s.stuck = true;
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
        s.stuck = true;
    }
    return s;
}

// Inclusive sum over the block's threads; *total receives the whole sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* part, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();   // part may still be read from the scan before
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int64_t p = part[w];
        if (w < warp) before += p;
        all += p;
    }
    *total = all;
    return x + before;
}

__global__ void __launch_bounds__(kThreads) gdn_kv_plan_kernel(const KvPlanArgs a) {
    __shared__ int64_t part[kWarps];
    __shared__ unsigned long long s_granted;
    __shared__ int s_len[kThreads], s_q[kThreads], s_held[kThreads], s_k0[kThreads];
    const unsigned rank = cluster_rank(), nrank = cluster_size();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool mine = warp % nrank == rank;       // this CTA copies this warp's sequences' pages
    const int tiles = (a.B + kThreads - 1) / kThreads;
    int status = 0;
    int count = *a.count_in;
    if (count < 0 || count > a.num_pages) {
        if (tid == 0) status |= kStatusBadLength;
        count = min(max(count, 0), a.num_pages);
    }
    if (tid == 0) s_granted = 0;

    // Returned pages onto the free list, in order of b and of the pages within b.
    Seq s = {};
    int64_t carry = count;
    for (int tile = 0; tile < tiles; ++tile) {
        const int b = tile * kThreads + tid;
        int st = 0;
        s = Seq{};
        if (b < a.B) s = read_seq(a, b, st);
        if (tiles == 1) status |= st;
        const int back = max(s.held - s.want, 0);
        int64_t total;
        const int64_t at = carry + block_scan(back, part, &total) - back;
        if (mine) {
            if (back <= kLanePages)
                for (int i = 0; i < back; ++i)
                    if (at + i < a.num_pages) a.free_list[at + i] = a.table[(size_t)b * a.max_pages + s.want + i];
            for (unsigned m = __ballot_sync(kFull, back > kLanePages); m; m &= m - 1) {
                const int src = __ffs(m) - 1;
                const int n = __shfl_sync(kFull, back, src), w0 = __shfl_sync(kFull, s.want, src);
                const int64_t to = __shfl_sync(kFull, at, src);
                const int32_t* row = a.table + (size_t)(b - lane + src) * a.max_pages + w0;
                for (int i = lane; i < n; i += 32)
                    if (to + i < a.num_pages) a.free_list[to + i] = row[i];
            }
        }
        carry += total;
    }
    const int64_t have = carry < a.num_pages ? carry : a.num_pages;
    cluster_sync();

    // Pages handed out from the top, in the same order, while they last; then the slots.
    carry = 0;
    for (int tile = 0; tile < tiles; ++tile) {
        const int b0 = tile * kThreads, b = b0 + tid;
        if (tiles > 1) {
            s = Seq{};
            if (b < a.B) s = read_seq(a, b, status);
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
        __syncthreads();
        if (mine) {
            const int take = granted ? need : 0;
            if (take <= kLanePages)
                for (int i = 0; i < take; ++i)
                    a.table[(size_t)b * a.max_pages + s.held + i] = a.free_list[have - 1 - k0 - i];
            for (unsigned m = __ballot_sync(kFull, take > kLanePages); m; m &= m - 1) {
                const int src = __ffs(m) - 1;
                const int n = __shfl_sync(kFull, take, src), h0 = __shfl_sync(kFull, s.held, src);
                const int k = __shfl_sync(kFull, k0, src);
                int32_t* row = a.table + (size_t)(b - lane + src) * a.max_pages + h0;
                for (int i = lane; i < n; i += 32) row[i] = a.free_list[have - 1 - k - i];
            }
        }
        // A new page's id is read from the free list itself, so a slot waits for no table write.
        const unsigned n = (unsigned)min(kThreads, a.B - b0);
        const unsigned T = (unsigned)a.T, page = (unsigned)a.page;
        int64_t* slots = a.slots + (size_t)b0 * T;
        for (unsigned i = rank * kThreads + tid; i < n * T; i += nrank * kThreads) {   // n T <= 2^29
            const unsigned j = i / T, t = i - j * T;
            int64_t slot = -1;
            if ((int)t < s_q[j]) {
                const unsigned pos = (unsigned)s_len[j] + t, pg = pos / page;
                const int id = (int)pg < s_held[j] ? a.table[(size_t)(b0 + j) * a.max_pages + pg]
                                                   : a.free_list[have - 1 - s_k0[j] - ((int)pg - s_held[j])];
                slot = (int64_t)id * page + (pos - pg * page);
            }
            slots[i] = slot;
        }
        // The counts may be written in place: every CTA has read this tile's by now.
        cluster_sync();
        if (rank == 0 && b < a.B) {
            a.seq_out[b] = s.seq_out;
            a.held_out[b] = now;
            a.kv_len[b] = s.len + q;
            a.q_len[b] = q;
        }
    }
    if (rank == 0) {
        if (tid == 0) *a.count_out = (int)(have - (int64_t)s_granted);
        if (a.status_word) {
            status = __reduce_or_sync(kFull, status);
            if (lane == 0 && status) atomicOr(a.status_word, status);
        }
    }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
    const bool one = (int64_t)a.B * a.T <= kOneCtaSlots;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(one ? 1 : kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = one ? 1 : kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_kv_plan_kernel, a);
}

}  // namespace gdn
