// pages.cu -- next rows of a page table out of the present ones (idx_pages_update), and copies of pages (idx_pages_copy).
//
// shares counts a page's holders beyond the first, so a page that the free list gives out needs no entry. The update
//   1. takes one holder from every page of the present rows and adds one for every page that a next row keeps;
//   2. looks at the next rows' last pages that are not full, which their rows will write: one with another holder is replaced
//      by a fresh page and a copy order, but for the first of rows that all end in it;
//   3. numbers the fresh pages (a prefix sum over the rows) and writes the rows; what a replaced page or a refused row
//      held is taken back;
//   4. collects the pages whose count fell below zero, in page order, behind what is left of the free list.
// The steps depend on one another through counts that any row may change, so they are phases of one cluster with its
// barrier between them (counts are whole numbers: the order of the atomics does not show). A present row's first heir
// keeps its holders, so rows that merely go on change no count.
//
// Measured in replayed graphs: 64 rows of up to 64 pages, 6000 pages 10.8 us, 1024 rows of up to 250 pages that fork, shrink and
// end, 200,000 pages 23.4 us (3.1 MB; 63.6 with every holder counted twice, one load at a time and two passes over the pages). Both
// are chains of latencies: five barriers of 1100 to 1500 cycles, and between them two to four dependent loads, eight in flight a
// thread. Copies of pages: 54 us for 43 pages of 262 KB in 16
// layers, 6.7 TB/s read and written, the measured copy rate.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "pages_plan.h"

namespace cg = cooperative_groups;

namespace idx {

namespace {

constexpr int kThreadsP = 1024, kWarpsP = kThreadsP / 32;

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

// Dynamic shared memory: three words per next row (heirs and fresh pages take turns, heirs being one per present row), then a
// bitmap of kSegment pages.
constexpr int kSegment = 131072;
constexpr size_t pages_smem(int32_t n_out, int32_t B) {
    return (2 * (size_t)n_out + (size_t)(n_out > B ? n_out : B)) * sizeof(int32_t) + kSegment / 8;
}
static_assert(pages_smem(kPagesMaxRows, kPagesMaxRows) + (32 + kCtasMost) * sizeof(int32_t) <= 227 * 1024,
              "with the kernel's static arrays within a CTA's shared memory");

// put(j, get(j)) for j = first, first + step, .. below end, kBatch loads at a time in flight.
constexpr int kBatch = 8;
template <typename Get, typename Put>
__device__ __forceinline__ void in_batches(int first, int end, int step, Get get, Put put) {
    for (int j = first; j < end; j += kBatch * step) {
        int32_t x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) x[u] = j + u * step < end ? get(j + u * step) : 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (j + u * step < end) put(j + u * step, x[u]);
    }
}

__global__ void __launch_bounds__(kThreadsP) pages_update_kernel(const PagesArgs a) {
    extern __shared__ int32_t sm[];
    uint32_t* freed_bits = reinterpret_cast<uint32_t*>(sm);  // [kSegment / 32]
    int32_t* keeps = sm + kSegment / 32;                     // [n_out] pages that a next row keeps
    int32_t* part = keeps + a.n_out;                         // [n_out] a row's last page, where it is not full; -1
    int32_t* heir = part + a.n_out;                          // [B] the first next row that continues a present one
    int32_t* fresh = heir;                                   // [n_out] entry of the free list; -1: none wanted, -2: none left
    __shared__ int warp_sums[32];
    __shared__ int freed[kCtasMost];  // pages that each CTA has found
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int all = ctas * kThreadsP, me = rank * kThreadsP + tid;     // threads of the cluster
    const int warps = ctas * kWarpsP, my_warp = warp * ctas + rank;    // its warps, neighbours on unlike SMs
    const int P = a.page_size;
    pdl_wait();
    pdl_launch_dependents();  // the kernel that only waits for this one

    auto pages_of = [&](int32_t len, int32_t width) -> int {  // of a row of len tokens; -1 where that breaks its bounds
        return len < 0 || len > (int64_t)width * P ? -1 : (int)(((int64_t)len + P - 1) / P);
    };
    auto add = [&](int32_t page, int by) {
        if ((uint32_t)page < (uint32_t)a.num_pages)
            atomicAdd(a.new_shares + page, by);
        else
            report(a.dev_status, IDX_STATUS_BAD_PAGE);
    };

    // ---- the rows, in every CTA alike ------------------------------------------------------------------
    for (int i = tid; i < a.B; i += kThreadsP) heir[i] = INT32_MAX;
    __syncthreads();
    for (int b = tid; b < a.n_out; b += kThreadsP) {
        const int32_t p = a.parent[b], k = a.keep[b];
        int n = p < 0 && k == 0 ? 0 : -1;
        int32_t page = -1;
        if (p >= 0 && p < a.B && k >= 0) {
            const int32_t len = a.lens[p];
            if (pages_of(len, a.pt_stride) >= 0 && k <= len) n = pages_of(k, a.new_stride);
            if (n > 0) {
                atomicMin(heir + p, b);
                if (k % P) page = a.page_table[(int64_t)p * a.pt_stride + n - 1];
            }
        }
        if (n < 0 && rank == 0) report(a.dev_status, IDX_STATUS_BAD_LEN);
        keeps[b] = max(n, 0);
        part[b] = (uint32_t)page < (uint32_t)a.num_pages ? page : -1;
    }
    if (a.new_shares != a.shares)
        in_batches(me, a.num_pages, all, [&](int p) { return a.shares[p]; }, [&](int p, int32_t x) { a.new_shares[p] = x; });
    cluster.sync();

    // ---- 1: holders. What a row's first heir keeps stays held; the rest of it is released, other heirs hold it too ----
    for (int i = my_warp; i < a.B; i += warps) {
        const int n = pages_of(a.lens[i], a.pt_stride);
        if (n < 0 && lane == 0) report(a.dev_status, IDX_STATUS_BAD_LEN);
        const int32_t* row = a.page_table + (int64_t)i * a.pt_stride;
        in_batches((heir[i] < INT32_MAX ? keeps[heir[i]] : 0) + lane, n, 32, [&](int j) { return row[j]; },
                [&](int, int32_t page) { add(page, -1); });
    }
    for (int b = my_warp; b < a.n_out; b += warps) {
        const int n = keeps[b], p = n ? a.parent[b] : 0;
        if (n == 0 || heir[p] == b) continue;
        const int32_t* row = a.page_table + (int64_t)p * a.pt_stride;
        in_batches(lane, n, 32, [&](int j) { return row[j]; }, [&](int, int32_t page) { add(page, 1); });
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
    int head = a.free_span[0], tail = a.free_span[1];
    if (head < 0 || tail < head || tail > a.free_cap) {
        if (me == 0) report(a.dev_status, IDX_STATUS_BAD_PAGE);
        head = tail = 0;
    }
    cluster.sync();

    // ---- 3: fresh pages and the rows ------------------------------------------------------------------
    int taken = 0;
    for (int b0 = 0; b0 < a.n_out; b0 += kThreadsP) {
        const int b = b0 + tid;
        const bool copy = b < a.n_out && __ldcg(a.copies + 2 * b) >= 0;
        int n;
        const int at = head + taken + cta_sum(copy, warp_sums, n);
        if (b < a.n_out) fresh[b] = !copy ? -1 : at < tail ? at : -2;
        taken += n;
    }
    taken = min(taken, tail - head);
    __syncthreads();  // fresh[] is complete
    for (int b = my_warp; b < a.n_out; b += warps) {
        const int at = fresh[b], n = keeps[b];
        const int32_t* row = a.page_table + (int64_t)(n ? a.parent[b] : 0) * a.pt_stride;
        if (at == -2) {
            for (int j = lane; j < n; j += 32) add(row[j], -1);
            if (lane == 0) {
                report(a.dev_status, IDX_STATUS_NO_PAGE);
                a.new_lens[b] = 0;
            }
            continue;
        }
        int32_t* to = a.new_table + (int64_t)b * a.new_stride;
        if (lane == 0) {
            a.new_lens[b] = n > 0 ? a.keep[b] : 0;
            if (at >= 0) {
                const int32_t own = a.free_pages[at];
                if ((uint32_t)own >= (uint32_t)a.num_pages) report(a.dev_status, IDX_STATUS_BAD_PAGE);
                to[n - 1] = own;
                a.copies[2 * b + 1] = own;
                atomicAdd(a.new_shares + part[b], -1);
            }
        }
        in_batches(lane, at >= 0 ? n - 1 : n, 32, [&](int j) { return row[j]; }, [&](int j, int32_t page) {
            to[j] = page;
            if ((uint32_t)page >= (uint32_t)a.num_pages) report(a.dev_status, IDX_STATUS_BAD_PAGE);
        });
    }
    const int left = tail - head - taken;
    in_batches(me, min(left, a.new_free_cap), all, [&](int i) { return a.free_pages[head + taken + i]; },
               [&](int i, int32_t page) { a.new_free[i] = page; });
    cluster.sync();
    for (int b = my_warp; b < a.n_out; b += warps)  // every CTA has read the copies
        if (lane == 0 && fresh[b] == -2) a.copies[2 * b] = -1;

    // ---- 4: the free list ------------------------------------------------------------------------------
    // A CTA's pages, as many at a time as the bitmap holds: a warp takes 32 of them, eight loads in flight.
    const int per = ((a.num_pages + ctas - 1) / ctas + 31) / 32 * 32;
    const int p0 = min((int64_t)rank * per, (int64_t)a.num_pages), p1 = min((int64_t)p0 + per, (int64_t)a.num_pages);
    auto find = [&](int from, int end, bool clear) -> int {  // the CTA's count
        int n = 0;
        const int words = (end - from + 31) / 32;
        for (int w = warp; w < words; w += 8 * kWarpsP) {
            int32_t s[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int p = from + (w + u * kWarpsP) * 32 + lane;
                s[u] = w + u * kWarpsP < words && p < end ? __ldcg(a.new_shares + p) : 0;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const unsigned bits = __ballot_sync(kFull, s[u] < 0);
                if (w + u * kWarpsP < words) {
                    if (lane == 0) freed_bits[w + u * kWarpsP] = bits;
                    n += lane == 0 ? __popc(bits) : 0;
                    if (s[u] < 0 && clear) {
                        if (s[u] < -1) report(a.dev_status, IDX_STATUS_BAD_PAGE);  // held by more rows than its count says
                        a.new_shares[from + (w + u * kWarpsP) * 32 + lane] = 0;
                    }
                }
            }
        }
        int sum;
        cta_sum(n, warp_sums, sum);
        return sum;
    };
    const bool once = p1 - p0 <= kSegment;
    int mine = 0;
    for (int p = p0; p < p1; p += kSegment) mine += find(p, min(p1 - p, kSegment) + p, once);
    if (tid < ctas) *cluster.map_shared_rank(&freed[rank], tid) = mine;
    cluster.sync();
    int at = left, total = left;
    for (int c = 0; c < ctas; ++c) {
        total += freed[c];
        if (c < rank) at += freed[c];
    }
    for (int p = p0; mine > 0 && p < p1; p += kSegment) {
        const int end = min(p1 - p, kSegment) + p, words = (end - p + 31) / 32;
        if (!once) find(p, end, true);
        const int per_thread = (words + kThreadsP - 1) / kThreadsP;
        const int w0 = min(tid * per_thread, words), w1 = min(w0 + per_thread, words);
        int n = 0, sum;
        for (int w = w0; w < w1; ++w) n += __popc(freed_bits[w]);
        int to = at + cta_sum(n, warp_sums, sum);
        for (int w = w0; w < w1; ++w)
            for (uint32_t bits = freed_bits[w]; bits; bits &= bits - 1, ++to)
                if (to < a.new_free_cap) a.new_free[to] = p + 32 * w + __ffs(bits) - 1;
        at += sum;
        __syncthreads();  // the bitmap is used again
    }
    if (me == 0) {
        a.new_span[0] = 0;
        a.new_span[1] = min(total, a.new_free_cap);
    }
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

// Clusters of kCtasMost CTAs that the current device takes at once, with all the shared memory that a call may ask for. Asked
// once per device (64 at most are remembered).
int wide_clusters() {
    static std::atomic<uint64_t> known{0}, fit{0};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (known.load(std::memory_order_acquire) & bit) return (fit.load(std::memory_order_relaxed) & bit) != 0;
    cudaError_t e = cudaFuncSetAttribute(pages_update_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kCtasMost;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(kCtasMost);
        cfg.blockDim = dim3(kThreadsP);
        cfg.dynamicSmemBytes = pages_smem(kPagesMaxRows, kPagesMaxRows);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, pages_update_kernel, &cfg);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();  // the narrow cluster is launched all the same
        n = 0;
    }
    if (n > 0) fit.fetch_or(bit, std::memory_order_relaxed);
    known.fetch_or(bit, std::memory_order_release);
    return n;
}

}  // namespace

cudaError_t launch_pages_update(const PagesArgs& a, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(allowed, pages_update_kernel, (int)pages_smem(kPagesMaxRows, kPagesMaxRows));
    if (e != cudaSuccess) return e;
    const int64_t entries = (int64_t)a.B * a.pt_stride + (int64_t)a.n_out * a.new_stride + a.num_pages;
    const int ctas = pages_ctas(entries, wide_clusters);
    e = launch_cluster(pages_update_kernel, dim3(ctas), dim3(kThreadsP), ctas, pages_smem(a.n_out, a.B), st, a);
    return e == cudaSuccess ? launch_done(st) : e;  // the library's kernels read lengths and tables before they wait
}

cudaError_t launch_pages_copy(const CopyArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.page_bytes + kCopyBytes - 1) / kCopyBytes), (unsigned)a.n, (unsigned)a.layers);
    return launch_pdl(pages_copy_kernel, grid, dim3(kCopyThreads), 0, st, a);
}

}  // namespace idx
