// compact.cu -- accepted tokens of a drafting step moved together in the paged caches (idx_kv_compact, idx_k_compact).
//
// The token of node path[i] goes from position front + path[i] to front + i, front being the number of keys in front of the
// tree. Paths increase, so a token never moves up and what is written lies in front of everything that is still to be
// read: a warp takes a request's tokens in order, in pieces that it holds in registers between reading and writing.
//
// 8-bit KV cache: a piece is a destination block of 16 tokens, which share a scale. Its new exponent is the largest of the blocks
// that its tokens come from (its own too where it keeps tokens in front of the tree), and codes from blocks of a smaller one shift
// down by the difference: a power of two, so exact but for codes that become subnormal.
// Indexer's cache: scales belong to tokens, the bytes move as they are.
//
// A warp per request, head and layer (a lane has 16 bytes of two or four tokens): the chains of loads, lengths, path, page
// table, scales, rows, are what it takes, and there are many of them. In replayed graphs 64 requests of up to 6 tokens in 8 layers
// of 8 heads (4.8 MB moved) take 6.6 us, 64 of up to 9 in one layer of the indexer's cache 3.9, about 1 of it for the kernel that
// orders new_lens; a call from the host takes 10.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "kv.cuh"

namespace idx {

namespace {

struct Request {
    int32_t front, n;  // keys in front of the tree; accepted nodes, 0 where there is nothing to move
    int32_t len;       // the sequence's keys behind the call
};

// A warp reads a request's lengths and tests its path.
__device__ __forceinline__ Request request(const CompactArgs& a, int b, bool tell) {
    const int lane = threadIdx.x & 31;
    const int32_t c0 = a.cu_seqlens_q[b], c1 = a.cu_seqlens_q[b + 1], len = a.seq_lens_k[b], n = a.n_path[b];
    const int64_t nq = (int64_t)c1 - c0;
    Request r{0, 0, max(len, 0)};
    if (nq < 0 || len < 0 || len > (int64_t)a.pt_stride * a.page_size || n < 0 || n > nq || n > a.max_path) {
        if (tell && lane == 0) report(a.dev_status, IDX_STATUS_BAD_LEN);
        return r;
    }
    if (len < nq) return r;  // a request that got no room this step
    bool ok = true;
    for (int i = lane; i < n; i += 32) {
        const int32_t x = a.path[(int64_t)b * a.max_path + i], before = i ? a.path[(int64_t)b * a.max_path + i - 1] : -1;
        ok &= x > before && x < nq;
    }
    if (!__all_sync(kFull, ok)) {
        if (tell && lane == 0) report(a.dev_status, IDX_STATUS_BAD_VALUE);
        return r;
    }
    r.front = (int32_t)(len - nq);
    r.n = n;
    r.len = r.front + n;
    return r;
}

// 16 codes times 2^-down
__device__ __forceinline__ uint4 shift_codes(uint4 w, int down) {
    const float g = pow2f(-down);
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        e4m3x4_to_f16x4(u[j], lo, hi);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        u[j] = f32x2_to_e4m3x2(x.x * g, x.y * g) | f32x2_to_e4m3x2(y.x * g, y.y * g) << 16;
    }
    return w;
}
__device__ __forceinline__ int scale_of(uint32_t byte) {  // exponent + 127, as the readers take it
    return min(max((int)byte, 127 + kKvEMin), 127 + kKvEMax);
}

template <int D>
__global__ void __launch_bounds__(128) kv_compact_kernel(const CompactArgs a) {
    constexpr int kLanes = D / 8;              // lanes of a token, 16 bytes each: K, then V
    constexpr int kTokens = 32 / kLanes;       // tokens of one load
    constexpr int kSteps = kKvBlock / kTokens;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, c = lane % kLanes, sub = lane / kLanes, side = c >= kLanes / 2;
    const int head = blockIdx.y * 4 + (threadIdx.x >> 5), b = blockIdx.x, layer = blockIdx.z;
    if (head >= a.kv_heads) return;
    const bool tell = head == 0 && layer == 0;
    const Request rq = request(a, b, tell);
    if (tell && a.new_lens && lane == 0) a.new_lens[b] = rq.len;
    const int P = a.page_size;
    uint8_t* pool = a.pool + layer * a.layer_stride + head * kv_head_bytes(P, D);
    const int32_t* pt = a.page_table + (int64_t)b * a.pt_stride;
    const int32_t* path = a.path + (int64_t)b * a.max_path;
    bool bad = false;
    for (int i0 = 0; i0 < rq.n;) {
        const int d0 = rq.front + i0, f = d0 % kKvBlock;
        const int n = min(rq.n - i0, kKvBlock - f);
        const int held = i0 == 0 ? f : 0;  // tokens in front of the tree
        const int32_t to = pt[d0 / P];
        const bool to_ok = (uint32_t)to < (uint64_t)a.num_pages;
        uint8_t* block = pool + (int64_t)to * a.page_stride + (int64_t)(d0 % P - f) * 2 * D;
        uint8_t* scale = pool + (int64_t)to * a.page_stride + 2ll * P * D + 2 * (d0 % P / kKvBlock);
        // lane t looks after token t of the piece: where it is, and its block's scales
        int64_t from = -1;
        int ek = 0, ev = 0;
        bool moves = false;
        if (lane < n) {
            const int pos = rq.front + path[i0 + lane];
            const int32_t page = pt[pos / P];
            if ((uint32_t)page < (uint64_t)a.num_pages && to_ok) {
                from = (int64_t)page * a.page_stride + (int64_t)(pos % P) * 2 * D;
                const uint32_t two = *reinterpret_cast<const uint16_t*>(pool + (int64_t)page * a.page_stride + 2ll * P * D +
                                                                        2 * (pos % P / kKvBlock));
                ek = scale_of(two & 255);
                ev = scale_of(two >> 8);
                moves = path[i0 + lane] != i0 + lane;
            } else {
                bad = true;
            }
        }
        if (__any_sync(kFull, moves)) {
            int old_k = 0, old_v = 0;
            if (held) {
                const uint32_t two = *reinterpret_cast<const uint16_t*>(scale);
                old_k = scale_of(two & 255);
                old_v = scale_of(two >> 8);
            }
            const int top_k = max(old_k, (int)__reduce_max_sync(kFull, (unsigned)ek));
            const int top_v = max(old_v, (int)__reduce_max_sync(kFull, (unsigned)ev));
            const int top = side ? top_v : top_k;
            uint4 w[kSteps];
            int down[kSteps];
            bool in[kSteps];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int t = s * kTokens + sub;
                const int64_t at = __shfl_sync(kFull, from, t);
                const int k = __shfl_sync(kFull, ek, t), v = __shfl_sync(kFull, ev, t);
                down[s] = top - (side ? v : k);
                in[s] = t < n && at >= 0;
                if (in[s]) w[s] = *reinterpret_cast<const uint4*>(pool + at + 16 * c);
            }
            __syncwarp();  // every lane has read
            const int old = side ? old_v : old_k;
            if (held && top > old) {
                for (int t = sub; t < held; t += kTokens) {
                    uint4* at = reinterpret_cast<uint4*>(block + (int64_t)t * 2 * D + 16 * c);
                    *at = shift_codes(*at, top - old);
                }
            }
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                if (!in[s]) continue;
                const int t = f + s * kTokens + sub;
                *reinterpret_cast<uint4*>(block + (int64_t)t * 2 * D + 16 * c) = down[s] ? shift_codes(w[s], down[s]) : w[s];
            }
            if (lane == 0) *reinterpret_cast<uint16_t*>(scale) = (uint16_t)(top_k | top_v << 8);
            __syncwarp();
        }
        i0 += n;
    }
    if (bad) report(a.dev_status, IDX_STATUS_BAD_PAGE);
}

template <bool kFp8>
__global__ void __launch_bounds__(128) k_compact_kernel(const CompactArgs a) {
    constexpr int kLanes = kFp8 ? 8 : 4;   // 16-byte chunks of a token
    constexpr int kTokens = 32 / kLanes;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, c = lane % kLanes, sub = lane / kLanes;
    const int b = blockIdx.x * 4 + (threadIdx.x >> 5), layer = blockIdx.y;
    if (b >= a.B) return;
    const Request rq = request(a, b, layer == 0);
    if (layer == 0 && a.new_lens && lane == 0) a.new_lens[b] = rq.len;
    const int P = a.page_size;
    uint8_t* pool = a.pool + layer * a.layer_stride;
    const int32_t* pt = a.page_table + (int64_t)b * a.pt_stride;
    const int32_t* path = a.path + (int64_t)b * a.max_path;
    auto chunk = [&](int s) { return kFp8 ? f8_chunk_off(s, c) : mx_chunk_off(P, s, c); };
    auto scale = [&](int s) { return kFp8 ? f8_scale_off(P, s) : mx_scale_off(P, s); };
    bool bad = false;
    for (int i0 = 0; i0 < rq.n; i0 += kTokens) {
        const int i = i0 + sub;
        bool moves = false;
        uint4 w = make_uint4(0, 0, 0, 0);
        uint32_t sc = 0;
        uint8_t* to = nullptr;
        if (i < rq.n && path[i] != i) {
            const int src = rq.front + path[i], dst = rq.front + i;
            const int32_t ps = pt[src / P], pd = pt[dst / P];
            moves = (uint32_t)ps < (uint64_t)a.num_pages && (uint32_t)pd < (uint64_t)a.num_pages;
            bad |= !moves;
            if (moves) {
                const uint8_t* at = pool + (int64_t)ps * a.page_stride;
                to = pool + (int64_t)pd * a.page_stride;
                w = *reinterpret_cast<const uint4*>(at + chunk(src % P));
                sc = *reinterpret_cast<const uint32_t*>(at + scale(src % P));
            }
        }
        __syncwarp();  // every lane has read
        if (moves) {
            const int s = (rq.front + i) % P;
            *reinterpret_cast<uint4*>(to + chunk(s)) = w;
            if (c == 0) *reinterpret_cast<uint32_t*>(to + scale(s)) = sc;
        }
        __syncwarp();
    }
    if (bad) report(a.dev_status, IDX_STATUS_BAD_PAGE);
}

}  // namespace

cudaError_t launch_kv_compact(const CompactArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)a.B, (unsigned)((a.kv_heads + 3) / 4), (unsigned)a.layers);
    const cudaError_t e = a.head_dim == 128 ? launch_pdl(kv_compact_kernel<128>, grid, dim3(128), 0, st, a)
                                            : launch_pdl(kv_compact_kernel<64>, grid, dim3(128), 0, st, a);
    // the library's kernels read lengths before they wait for what is in front of them
    return e == cudaSuccess && a.new_lens ? launch_done(st) : e;
}

cudaError_t launch_k_compact(const CompactArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.B + 3) / 4), (unsigned)a.layers);
    const cudaError_t e = a.dtype == IDX_FP8 ? launch_pdl(k_compact_kernel<true>, grid, dim3(128), 0, st, a)
                                             : launch_pdl(k_compact_kernel<false>, grid, dim3(128), 0, st, a);
    return e == cudaSuccess && a.new_lens ? launch_done(st) : e;
}

}  // namespace idx
