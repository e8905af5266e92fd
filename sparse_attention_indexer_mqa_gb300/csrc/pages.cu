// pages.cu -- next rows of a page table out of the present ones (idx_pages_update), and copies of pages (idx_pages_copy).
//
// shares counts a page's holders beyond the first, so a page that the free list gives out needs no entry. The update
//   1. takes one holder from every page of the present rows and adds one for every page that a next row keeps;
//   2. looks at the next rows' last pages that are not full, which their rows will write: one with another holder is replaced
//      by a fresh page and a copy order, but for the first of rows that all end in it;
//   3. numbers the fresh pages (a prefix sum over the rows) and writes the rows; what a replaced page or a refused row
//      held is taken back;
//   4. collects the pages whose count fell below zero, in page order, behind what is left of the free list.
// The steps depend on one another through counts that any row may change, so they are phases of one cluster of eight
// CTAs with its barrier between them (counts are whole numbers: the order of the atomics does not show).
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace idx {

namespace {

constexpr int kCtas = 8, kThreadsP = 1024, kWarpsP = kThreadsP / 32;

// Exclusive sum over the CTA of one value per thread, and the total.
__device__ __forceinline__ int cta_sum(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    int s = warp_sums[lane];  // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, s, o);
        if (lane >= o) s += y;
    }
    total = __shfl_sync(kFull, s, 31);
    const int before = w > 0 ? __shfl_sync(kFull, s, w - 1) : 0;
    __syncthreads();  // warp_sums is used again
    return before + x - v;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreadsP) pages_update_kernel(const PagesArgs a) {
    extern __shared__ int32_t sm[];
    int32_t* part = sm;            // [n_out] a row's last page, where it is not full; -1
    int32_t* fresh = sm + a.n_out;  // [n_out] the row's entry of the free list; -1: none wanted, -2: none left
    __shared__ int warp_sums[32];
    __shared__ int freed;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster.block_rank();
    const int all = kCtas * kThreadsP, me = rank * kThreadsP + tid;   // threads of the cluster
    const int warps = kCtas * kWarpsP, my_warp = warp * kCtas + rank;  // its warps, neighbours on unlike SMs
    const int P = a.page_size;
    pdl_wait();
    pdl_launch_dependents();  // the kernel that only waits for this one

    auto held = [&](int i) -> int {  // pages of a present row
        const int32_t len = a.lens[i];
        return len < 0 || len > (int64_t)a.pt_stride * P ? -1 : (int)(((int64_t)len + P - 1) / P);
    };
    auto kept = [&](int b) -> int {  // pages that a next row keeps; -1: an empty row that breaks its bounds
        const int32_t p = a.parent[b], k = a.keep[b];
        if (p < 0) return k == 0 ? 0 : -1;
        if (p >= a.B || k < 0 || held(p) < 0 || k > a.lens[p]) return -1;
        const int n = (int)(((int64_t)k + P - 1) / P);
        return n > a.new_stride ? -1 : n;
    };
    auto add = [&](int32_t page, int by) {
        if ((uint32_t)page < (uint32_t)a.num_pages)
            atomicAdd(a.new_shares + page, by);
        else
            report(a.dev_status, IDX_STATUS_BAD_PAGE);
    };

    if (a.new_shares != a.shares)
        for (int p = me; p < a.num_pages; p += all) a.new_shares[p] = a.shares[p];
    cluster.sync();

    // ---- 1: holders ----------------------------------------------------------------------------------
    for (int i = my_warp; i < a.B; i += warps) {
        const int n = held(i);
        if (n < 0 && lane == 0) report(a.dev_status, IDX_STATUS_BAD_LEN);
        for (int j = lane; j < n; j += 32) add(a.page_table[(int64_t)i * a.pt_stride + j], -1);
    }
    for (int b = my_warp; b < a.n_out; b += warps) {
        const int n = kept(b);
        if (n < 0 && lane == 0) report(a.dev_status, IDX_STATUS_BAD_LEN);
        for (int j = lane; j < n; j += 32) add(a.page_table[(int64_t)a.parent[b] * a.pt_stride + j], 1);
    }
    for (int b = tid; b < a.n_out; b += kThreadsP) {
        const int n = kept(b);
        int32_t page = -1;
        if (n > 0 && a.keep[b] % P) {
            page = a.page_table[(int64_t)a.parent[b] * a.pt_stride + n - 1];
            if ((uint32_t)page >= (uint32_t)a.num_pages) page = -1;
        }
        part[b] = page;
    }
    cluster.sync();

    // ---- 2: which rows need a page of their own ------------------------------------------------------
    for (int b = my_warp; b < a.n_out; b += warps) {
        const int32_t page = part[b];
        bool copy = false;
        if (page >= 0) {
            const int holders = __ldcg(a.new_shares + page) + 1;
            if (holders > 1) {
                int same = 0, before = 0;
                for (int x = lane; x < a.n_out; x += 32) {
                    const bool hit = part[x] == page;
                    same += hit;
                    before += hit && x < b;
                }
                same = __reduce_add_sync(kFull, same);
                before = __reduce_add_sync(kFull, before);
                copy = holders != same || before > 0;
            }
        }
        if (lane == 0) {
            a.copies[2 * b] = copy ? page : -1;
            a.copies[2 * b + 1] = -1;
        }
    }
    cluster.sync();

    // ---- 3: fresh pages and the rows ------------------------------------------------------------------
    int head = a.free_span[0], tail = a.free_span[1];
    if (head < 0 || tail < head || tail > a.free_cap) {
        if (me == 0) report(a.dev_status, IDX_STATUS_BAD_PAGE);
        head = tail = 0;
    }
    int taken;
    {
        const int per = (a.n_out + kThreadsP - 1) / kThreadsP, b0 = min(tid * per, a.n_out), b1 = min(b0 + per, a.n_out);
        int n = 0;
        for (int b = b0; b < b1; ++b) n += __ldcg(a.copies + 2 * b) >= 0;
        int at = head + cta_sum(n, warp_sums, taken);
        for (int b = b0; b < b1; ++b) {
            const bool copy = __ldcg(a.copies + 2 * b) >= 0;
            fresh[b] = !copy ? -1 : at < tail ? at : -2;
            at += copy;
        }
        taken = min(taken, tail - head);
    }
    if (tid == 0) freed = 0;
    cluster.sync();  // fresh[] is complete, and every CTA has read the copies
    for (int b = my_warp; b < a.n_out; b += warps) {
        const int at = fresh[b], n = max(kept(b), 0);
        const int32_t* row = a.page_table + (int64_t)a.parent[b] * a.pt_stride;
        if (at == -2) {
            for (int j = lane; j < n; j += 32) add(row[j], -1);
            if (lane == 0) {
                report(a.dev_status, IDX_STATUS_NO_PAGE);
                a.new_lens[b] = 0;
                a.copies[2 * b] = -1;
            }
            continue;
        }
        const int32_t own = at >= 0 ? a.free_pages[at] : -1;
        for (int j = lane; j < n; j += 32) a.new_table[(int64_t)b * a.new_stride + j] = at >= 0 && j == n - 1 ? own : row[j];
        if (lane == 0) {
            a.new_lens[b] = n > 0 ? a.keep[b] : 0;
            if (at >= 0) {
                if ((uint32_t)own >= (uint32_t)a.num_pages) report(a.dev_status, IDX_STATUS_BAD_PAGE);
                a.copies[2 * b + 1] = own;
                atomicAdd(a.new_shares + part[b], -1);
            }
        }
    }
    cluster.sync();

    // ---- 4: the free list ------------------------------------------------------------------------------
    const int per = (a.num_pages + kCtas - 1) / kCtas, p0 = min(rank * per, a.num_pages), p1 = min(p0 + per, a.num_pages);
    int n = 0;
    for (int p = p0 + tid; p < p1; p += kThreadsP) n += __ldcg(a.new_shares + p) < 0;
    int mine;
    cta_sum(n, warp_sums, mine);
    if (tid == 0) freed = mine;
    cluster.sync();
    const int left = tail - head - taken;
    int at = left, total = left;
    for (int c = 0; c < kCtas; ++c) {
        const int x = *cluster.map_shared_rank(&freed, c);
        total += x;
        if (c < rank) at += x;
    }
    for (int p = p0; mine > 0 && p < p1; p += kThreadsP) {
        const int32_t s = p + tid < p1 ? __ldcg(a.new_shares + p + tid) : 0;
        int sum;
        const int before = cta_sum(s < 0, warp_sums, sum);
        if (s < 0) {
            if (s < -1) report(a.dev_status, IDX_STATUS_BAD_PAGE);  // held by more rows than its count says
            if (at + before < a.new_free_cap) a.new_free[at + before] = p + tid;
            a.new_shares[p + tid] = 0;
        }
        at += sum;
    }
    for (int i = me; i < left && i < a.new_free_cap; i += all) a.new_free[i] = a.free_pages[head + taken + i];
    if (me == 0) {
        a.new_span[0] = 0;
        a.new_span[1] = min(total, a.new_free_cap);
    }
    cluster.sync();  // nobody reads another CTA's count any more
}

// 16 bytes a thread, eight of them in flight.
constexpr int kCopyThreads = 256, kCopyEach = 8, kCopyBytes = kCopyThreads * kCopyEach * 16;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CopyArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int pair = blockIdx.y, layer = blockIdx.z;
    const int32_t src = a.copies[2 * pair], dst = a.copies[2 * pair + 1];
    if (src < 0 || dst < 0 || src == dst) return;
    if (src >= a.num_pages || dst >= a.num_pages) {
        if (threadIdx.x == 0 && layer == 0 && blockIdx.x == 0) report(a.dev_status, IDX_STATUS_BAD_PAGE);
        return;
    }
    const uint4* from = reinterpret_cast<const uint4*>(a.pool + layer * a.layer_stride + src * a.page_stride);
    uint4* to = reinterpret_cast<uint4*>(a.pool + layer * a.layer_stride + dst * a.page_stride);
    const int64_t n = a.page_bytes / 16, at = (int64_t)blockIdx.x * (kCopyThreads * kCopyEach) + threadIdx.x;
    uint4 w[kCopyEach];
#pragma unroll
    for (int i = 0; i < kCopyEach; ++i)
        if (at + i * kCopyThreads < n) w[i] = from[at + i * kCopyThreads];
#pragma unroll
    for (int i = 0; i < kCopyEach; ++i)
        if (at + i * kCopyThreads < n) to[at + i * kCopyThreads] = w[i];
}

}  // namespace

cudaError_t launch_pages_update(const PagesArgs& a, cudaStream_t st) {
    const size_t smem = 2 * (size_t)a.n_out * sizeof(int32_t);
    if (smem > 48 * 1024) {  // raised to the most that any call needs: another thread's call may come in between
        static std::atomic<uint64_t> allowed{0};
        const cudaError_t s = allow_smem(allowed, pages_update_kernel, 2 * kPagesMaxRows * (int)sizeof(int32_t));
        if (s != cudaSuccess) return s;
    }
    const cudaError_t e = launch_pdl(pages_update_kernel, dim3(kCtas), dim3(kThreadsP), smem, st, a);
    return e == cudaSuccess ? launch_done(st) : e;  // the library's kernels read lengths and tables before they wait
}

cudaError_t launch_pages_copy(const CopyArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.page_bytes + kCopyBytes - 1) / kCopyBytes), (unsigned)a.n, (unsigned)a.layers);
    return launch_pdl(pages_copy_kernel, grid, dim3(kCopyThreads), 0, st, a);
}

}  // namespace idx
