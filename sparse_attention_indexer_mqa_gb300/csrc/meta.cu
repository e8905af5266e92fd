// meta.cu -- page tables, slot map, positions and lengths of a step from the requests' lengths
// (idx_step_meta).
//
// Two exclusive prefix sums over the requests give everything: of the new tokens (a request's
// first row) and of the new pages (its first entry of the free list). The pages' sum runs over
// the requests that passed the first one's checks. Every CTA takes both sums over all requests
// itself (8 bytes a request from L2, at most 16384 of them) and then writes its own rows and
// requests, so that no CTA waits for another. A row finds its
// request by binary search in the sums, which stay in shared memory (8 bytes a request).
// Reads and writes of the page table never meet: a row reads entries below ceil(ctx/P) or
// the free list, and only entries from ceil(ctx/P) on are written.
// Measured in a replayed graph: 64 requests of one token 6.0 us, 512 requests with 66173 rows 8.5 us (0.8 MB): launch,
// two sums with four barriers, and per row a binary search and two dependent loads; 0.4 and 0.7 us of it are the
// waiting kernel behind. A call from the host takes 10.6 and 11.0 us, 1.8 of them for the second launch.
#include "common.cuh"
#include "kernels.h"

namespace idx {

namespace {

// Exclusive sum over the CTA of one value per thread, and the total.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t* warp_sums, int64_t& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    int64_t s = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, s, o);
        if (lane >= o) s += y;
    }
    total = __shfl_sync(kFull, s, 31);
    const int64_t before = __shfl_sync(kFull, s, w > 0 ? w - 1 : 0);
    __syncthreads();  // warp_sums is used again
    return (w > 0 ? before : 0) + x - v;
}

__global__ void step_meta_kernel(const MetaArgs a, int rows_per_cta) {
    extern __shared__ int32_t sm[];
    int32_t* start = sm;              // [B + 1] first row of each request, at most T_cap
    int32_t* first = sm + a.B + 1;    // [B] first free-list entry; -1: the request gets nothing
    __shared__ int64_t warp_sums[32];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int per = (a.B + nt - 1) / nt;  // consecutive requests of a thread
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    const int64_t P = a.page_size;
    pdl_launch_dependents();  // step_meta_done_kernel

    int64_t head = a.free_span[0], tail = a.free_span[1];
    if (head < 0 || tail < head || tail > a.free_cap) {
        if (blockIdx.x == 0 && tid == 0) report(a.dev_status, IDX_STATUS_BAD_PAGE);
        head = head < 0 ? 0 : (head > a.free_cap ? a.free_cap : head);
        tail = head;
    }

    int64_t rows = 0, total;
    for (int b = b0; b < b1; ++b) rows += max(a.q_lens[b], 0);
    int64_t at = cta_scan(rows, warp_sums, total);
    int64_t pages = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t ctx = a.ctx_lens[b], q = a.q_lens[b], end = at + (q > 0 ? q : 0);
        const bool ok = ctx >= 0 && q >= 0 && ctx + q <= a.max_seq_len_k && end <= a.T_cap;
        start[b] = (int32_t)(at < a.T_cap ? at : a.T_cap);
        first[b] = ok ? 0 : -1;
        if (ok) pages += (ctx + q + P - 1) / P - (ctx + P - 1) / P;
        if (!ok && blockIdx.x == 0) report(a.dev_status, IDX_STATUS_BAD_LEN);
        at = end;
    }
    if (tid == 0) start[a.B] = (int32_t)(total < a.T_cap ? total : a.T_cap);
    at = head + cta_scan(pages, warp_sums, total);
    int64_t taken = head;  // where the demand up to this thread's last request that was not refused ends
    for (int b = b0; b < b1; ++b) {
        if (first[b] < 0) continue;
        const int64_t ctx = a.ctx_lens[b], q = a.q_lens[b];
        const int64_t need = (ctx + q + P - 1) / P - (ctx + P - 1) / P;
        if (need > 0 && at + need > tail) {
            first[b] = -1;
            if (blockIdx.x == 0) report(a.dev_status, IDX_STATUS_NO_PAGE);
        } else {
            if (need > 0) first[b] = (int32_t)at;
            taken = at + need;
        }
        at += need;
    }
    // the sums grow with the request, so the largest end is the last request's that was not refused
    if (blockIdx.x == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int64_t y = __shfl_xor_sync(kFull, taken, o);
            taken = y > taken ? y : taken;
        }
        if ((tid & 31) == 0) warp_sums[tid >> 5] = taken;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        for (int w = 1; w < (nt >> 5); ++w) taken = warp_sums[w] > taken ? warp_sums[w] : taken;
        *a.free_next = (int32_t)(taken < INT32_MAX ? taken : INT32_MAX);
        a.cu_seqlens_q[a.B] = start[a.B];
    }

    // this CTA's requests: lengths, prefix sums and the appended pages
    for (int b = blockIdx.x * nt + tid; b < a.B; b += gridDim.x * nt) {
        const bool ok = first[b] >= 0;
        const int64_t ctx = a.ctx_lens[b], len = ok ? ctx + a.q_lens[b] : 0;
        a.cu_seqlens_q[b] = start[b];
        a.seq_lens_k[b] = (int32_t)len;
        if (!ok) continue;
        const int64_t j0 = (ctx + P - 1) / P, j1 = (len + P - 1) / P;
        for (int64_t j = j0; j < j1; ++j) {
            const int32_t page = a.free_pages[first[b] + (j - j0)];
            if ((uint32_t)page >= (uint64_t)a.num_pages) report(a.dev_status, IDX_STATUS_BAD_PAGE);
            a.page_table[(int64_t)b * a.pt_stride + j] = page;
        }
    }

    // this CTA's rows
    const int32_t live = start[a.B];
    const int64_t r0 = (int64_t)blockIdx.x * rows_per_cta;
    for (int64_t t = r0 + tid; t < r0 + rows_per_cta && t < a.T_cap; t += nt) {
        int64_t slot = -1;
        int32_t pos = 0;
        if (t < live) {
            int lo = 0, hi = a.B;  // the last request that starts at or before row t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start[mid] <= t) lo = mid; else hi = mid;
            }
            if (first[lo] >= 0) {
                const int64_t ctx = a.ctx_lens[lo], p = ctx + (t - start[lo]);
                const int64_t j = p / P, j0 = (ctx + P - 1) / P;
                const int32_t page =
                    j < j0 ? a.page_table[(int64_t)lo * a.pt_stride + j] : a.free_pages[first[lo] + (j - j0)];
                pos = (int32_t)p;
                if ((uint32_t)page < (uint64_t)a.num_pages)
                    slot = page * P + p % P;
                else
                    report(a.dev_status, IDX_STATUS_BAD_PAGE);
            }
        }
        a.positions[t] = pos;
        a.slot_mapping[t] = slot;
    }
}

// Behind the metadata: returns when they are visible. The library's kernels read lengths and page tables before they
// wait for the kernel in front of them, and a kernel launched with programmatic serialization may start as
// soon as the CTAs of that one have ended. In front of them is this one, whose CTA ends behind its wait: whatever
// is launched next, eagerly, captured or replayed, starts when the metadata are there. It is resident while the
// metadata kernel runs.
__global__ void step_meta_done_kernel() { pdl_wait(); }

}  // namespace

cudaError_t launch_step_meta(const MetaArgs& a, cudaStream_t st) {
    // a thread per request for the sums where that fits, and a thread per row (512 requests, 66173 rows: 7.8 us, 11.8
    // with four rows a thread, the waiting kernel not counted)
    const int threads = a.B <= 256 ? 256 : 1024;
    const int rows = threads;
    const int64_t ctas = a.T_cap > rows ? (a.T_cap + rows - 1) / rows : 1;
    const size_t smem = (2 * (size_t)a.B + 1) * sizeof(int32_t);
    if (smem > 48 * 1024) {  // raised to the most that any call needs: another thread's call may come in between
        static std::atomic<uint64_t> allowed{0};
        const cudaError_t s = allow_smem(allowed, step_meta_kernel, (2 * kMetaMaxRequests + 1) * (int)sizeof(int32_t));
        if (s != cudaSuccess) return s;
    }
    const cudaError_t e = launch_k(false, step_meta_kernel, dim3((unsigned)ctas), dim3(threads), smem, st, a, rows);
    return e == cudaSuccess ? launch_pdl(step_meta_done_kernel, dim3(1), dim3(32), 0, st) : e;
}

}  // namespace idx
