// verify.cu -- the walk through a tree of drafted tokens (idx_draft_verify).
//
// A walk stands on a node (first the root) and tests its children in index order. With the drafter's probabilities q,
// from which all children of a node were drawn independently, the target's p and k children rejected so far, the next
// is accepted with the chance min(1, p_k(x) / q(x)), where p_0 = p and p_{k+1} = max(p_k - q, 0) / Z_k. By induction
//     p_k = max(p - c_k q, 0) / S_k,   c_0 = 0, S_0 = 1,   c_{k+1} = c_k + S_k,   S_k = sum over the vocabulary of max(p - c_k q, 0),
// so a rejection costs one pass over the two rows and nothing is stored. Without q (children chosen, not drawn: point
// masses) p_{k+1} is p_k without x: S falls by p(x), and a bit per token says what is left. Where no child is left, a token is drawn
// from p_k: the first one whose running sum passes r times the row's sum.
// Sums are 64-bit: the draw looks for a border among a vocabulary's running sums, and with 2^17 of them an error of 2^-24 in each
// would move one draw in a hundred.
//
// A CTA per request; all its threads follow the walk, and share the passes over a row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace idx {

namespace {

constexpr int kThreadsV = 1024, kWarpsV = kThreadsV / 32;

template <typename T>
__device__ __forceinline__ float prob(const T* row, int i);
template <>
__device__ __forceinline__ float prob<float>(const float* row, int i) { return row[i]; }
template <>
__device__ __forceinline__ float prob<__nv_bfloat16>(const __nv_bfloat16* row, int i) { return __bfloat162float(row[i]); }
template <>
__device__ __forceinline__ float prob<__half>(const __half* row, int i) { return __half2float(row[i]); }

// What is no probability (negative, NaN, infinite) counts as zero.
__device__ __forceinline__ float clean(float x, bool& bad) {
    const bool ok = x >= 0.0f && x < __int_as_float(0x7f800000);
    bad |= !ok;
    return ok ? x : 0.0f;
}

template <typename T, bool kDrafter>
__global__ void __launch_bounds__(kThreadsV) draft_verify_kernel(const VerifyArgs a) {
    extern __shared__ uint32_t gone[];  // without a drafter: a bit per token that was rejected at the node
    __shared__ double sums[kWarpsV];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const int32_t c0 = a.cu_seqlens_q[b], c1 = a.cu_seqlens_q[b + 1], n = c1 - c0;
    const bool fine = c0 >= 0 && c1 >= c0 && c1 <= a.T && n <= a.max_q_len;
    int32_t* path = a.path + (int64_t)b * a.max_path;
    int32_t* out = a.out_tokens + (int64_t)b * a.max_path;
    for (int i = tid; i < a.max_path; i += kThreadsV) {
        path[i] = fine && n > 0 && i == 0 ? 0 : -1;
        out[i] = -1;
    }
    if (!fine || n == 0) {
        if (tid == 0) {
            a.n_path[b] = 0;
            if (!fine) report(a.dev_status, IDX_STATUS_BAD_LEN);
        }
        return;
    }
    const int words = (a.V + 31) / 32;
    if constexpr (!kDrafter) {
        for (int i = tid; i < words; i += kThreadsV) gone[i] = 0;
    }
    __syncthreads();

    const int32_t* tokens = a.tokens + c0;
    const int32_t* parents = a.parents + c0;
    const float* coins = a.coins + c0;
    int cur = 0, length = 1, rejected = 0;
    double cut = 0.0, mass = 1.0;
    bool bad = false, bad_token = false;
    const T* p = static_cast<const T*>(a.target) + (int64_t)c0 * a.target_stride;
    const T* q = kDrafter ? static_cast<const T*>(a.draft) + (int64_t)c0 * a.draft_stride : nullptr;

    // what is left of token v's probability
    auto left = [&](int v, double with_cut) -> double {
        const float x = clean(prob(p, v), bad);
        if constexpr (kDrafter) {
            if (with_cut == 0.0) return x;
            const double w = (double)x - with_cut * (double)clean(prob(q, v), bad);
            return w > 0.0 ? w : 0.0;
        } else {
            return (gone[v >> 5] >> (v & 31)) & 1u ? 0.0 : (double)x;
        }
    };
    // a warp's part of the vocabulary, and its sum; the sum over all of them
    const int part = (a.V + kWarpsV - 1) / kWarpsV, v0 = min(warp * part, a.V), v1 = min(v0 + part, a.V);
    auto total = [&](auto&& weight) -> double {
        double s = 0.0;
        for (int v = v0 + lane; v < v1; v += 32) s += weight(v);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        __syncthreads();  // the last sums have been read
        if (lane == 0) sums[warp] = s;
        __syncthreads();
        double t = 0.0;
        for (int w = 0; w < kWarpsV; ++w) t += sums[w];
        return t;
    };

    for (int j = 1; length < a.max_path;) {
        // the next child, found by each warp for itself
        int child = -1;
        for (; j < n; j += 32) {
            const unsigned hit = __ballot_sync(kFull, j + lane < n && parents[j + lane] == cur);
            if (hit) {
                child = j + __ffs(hit) - 1;
                break;
            }
        }
        if (child < 0) break;
        j = child + 1;
        const int x = tokens[child];
        if (x < 0 || x >= a.V) {
            bad_token = true;
            continue;
        }
        const double u = coins[child];
        bool yes;
        if constexpr (kDrafter) {
            const double px = clean(prob(p, x), bad), qx = clean(prob(q, x), bad);
            yes = __dmul_rn(__dmul_rn(u, qx), mass) < __dsub_rn(px, __dmul_rn(cut, qx));
            if (!yes) {
                cut += mass;
                const double by = cut;
                mass = total([&](int v) { return left(v, by); });
            }
        } else {
            const double px = (gone[x >> 5] >> (x & 31)) & 1u ? 0.0 : (double)clean(prob(p, x), bad);
            yes = __dmul_rn(u, mass) < px;
            if (!yes) mass = mass > px ? mass - px : 0.0;
            __syncthreads();  // every warp has read the bit
            if (!yes && tid == 0) gone[x >> 5] |= 1u << (x & 31);
            __syncthreads();
        }
        if (!yes) {
            ++rejected;
            continue;
        }
        if (tid == 0) {
            path[length] = child;
            out[length - 1] = x;
        }
        ++length;
        if (!kDrafter && rejected) {
            for (int i = tid; i < words; i += kThreadsV) gone[i] = 0;
            __syncthreads();
        }
        cur = child;
        cut = 0.0;
        mass = 1.0;
        rejected = 0;
        p = static_cast<const T*>(a.target) + (int64_t)(c0 + cur) * a.target_stride;
        if constexpr (kDrafter) q = static_cast<const T*>(a.draft) + (int64_t)(c0 + cur) * a.draft_stride;
    }

    // ---- the draw ------------------------------------------------------------------------------------
    bool whole = false;  // nothing is left of p: p itself
    auto weight = [&](int v) -> double { return whole ? (double)clean(prob(p, v), bad) : left(v, cut); };
    double all = total(weight);
    if (!(all > 0.0)) {
        whole = true;
        all = total(weight);
    }
    float r = a.last[b];
    const bool bad_coin = !(r >= 0.0f && r < 1.0f);
    if (!(r >= 0.0f)) r = 0.0f;
    const double goal = __dmul_rn((double)r, all);
    // the warp whose part holds the border; with r >= 1 the last that holds anything
    int at = -1;
    double before = 0.0, run = 0.0;
    for (int w = 0; w < kWarpsV; ++w) {
        if (sums[w] > 0.0) {
            at = w;
            before = run;
        }
        run += sums[w];
        if (run > goal) break;
    }
    if (warp == max(at, 0)) {
        int found = -1;
        double s = before;
        for (int v = v0; v < v1; v += 32) {
            const double w = v + lane < v1 ? weight(v + lane) : 0.0;
            double x = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            const unsigned pass = __ballot_sync(kFull, w > 0.0 && s + x > goal);
            const unsigned some = __ballot_sync(kFull, w > 0.0);
            if (pass) {
                found = v + __ffs(pass) - 1;
                break;
            }
            if (some) found = v + 31 - __clz(some);
            s += __shfl_sync(kFull, x, 31);
        }
        if (lane == 0) {
            out[length - 1] = found;
            a.n_path[b] = length;
            if (found < 0 || bad_coin || bad_token) report(a.dev_status, IDX_STATUS_BAD_VALUE);
        }
    }
    if (bad) report(a.dev_status, IDX_STATUS_BAD_VALUE);
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)a.B), block(kThreadsV);
    if (a.draft) return launch_pdl(draft_verify_kernel<T, true>, grid, block, 0, st, a);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(allowed, draft_verify_kernel<T, false>, kVerifyMaxVocab / 8);
    if (e != cudaSuccess) return e;
    return launch_pdl(draft_verify_kernel<T, false>, grid, block, (size_t)((a.V + 31) / 32) * 4, st, a);
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyArgs& a, cudaStream_t st) {
    if (a.ptype == IDX_FP32) return launch<float>(a, st);
    return a.ptype == IDX_BF16 ? launch<__nv_bfloat16>(a, st) : launch<__half>(a, st);
}

}  // namespace idx
