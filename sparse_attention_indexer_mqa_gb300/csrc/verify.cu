// verify.cu -- the walk through a tree of drafted tokens (idx_draft_verify).
//
// A walk stands on a node (first the root) and tests its children in index order. With the drafter's probabilities q,
// from which all children of a node were drawn independently, the target's p and k children rejected so far, the next
// is accepted with the chance min(1, p_k(x) / q(x)), where p_0 = p and p_{k+1} = max(p_k - q, 0) / Z_k. By induction
//     p_k = max(p - c_k q, 0) / S_k,   c_0 = 0, S_0 = 1,   c_{k+1} = c_k + S_k,   S_k = sum over the vocabulary of max(p - c_k q, 0),
// so a rejection costs one pass over the two rows and nothing is stored. Without q (children chosen, not drawn: point
// masses) p_{k+1} is p_k without x: S falls by p(x). Where no child is left, a token is drawn from p_k: the first one whose
// running sum passes r times the row's sum. The last rejection's pass has left the sums that the search starts from.
//
// Sums. The draw looks for a border among a vocabulary's running sums, and with 2^17 of them an error of 2^-24 in each
// would move one draw in a hundred. fp64 has a 64th of fp32's rate here, so weights and sums are pairs of fp32 (a
// value and what its rounding lost, by error-free sums and products), about 2^-46 of the sum; only the few totals
// and the search inside one warp's part are fp64.
//
// A cluster of eight CTAs per request: the row is cut into eight slices, a slice into the CTA's warps' parts. All
// threads follow the walk by themselves; a pass ends with one cluster barrier, behind which every CTA adds up the
// eight totals in the same order. What the walk asks of each node (its parent, token, number and the two
// probabilities) is fetched for 256 nodes at once, so that a step between passes is no chain of loads.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace idx {

namespace {

constexpr int kCtasV = 8, kThreadsV = 256, kWarpsV = kThreadsV / 32;
constexpr int kNodes = kThreadsV;  // nodes that are staged at once

// A sum and what its roundings lost.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ void add(Pair& s, float x) {  // s.hi + x exactly, as a sum and its error
    const float t = __fadd_rn(s.hi, x), b = __fsub_rn(t, s.hi);
    s.lo += __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x, b));
    s.hi = t;
}
__device__ __forceinline__ void add(Pair& s, const Pair& x) {
    add(s, x.hi);
    s.lo += x.lo;
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// What is no probability (negative, NaN, infinite) counts as zero.
__device__ __forceinline__ float clean(float x, bool& bad) {
    const bool ok = x >= 0.0f && x < __int_as_float(0x7f800000);
    bad |= !ok;
    return ok ? x : 0.0f;
}

// Vectors of a row: 16 bytes each where the row's address allows; vector k holds elements k * kVec - off ..
template <typename T>
struct Row {
    static constexpr int kVec = 16 / sizeof(T);
    const T* at;
    __device__ __forceinline__ int off() const { return (int)((reinterpret_cast<uintptr_t>(at) / sizeof(T)) % kVec); }
};

// Elements e0 .. e0 + kVec - 1 of a row of V; those outside it are 0. whole: e0 lies on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load(const T* row, int e0, int V, bool whole, bool& bad, float (&x)[16 / sizeof(T)]) {
    constexpr int kVec = 16 / sizeof(T);
    if (whole && e0 >= 0 && e0 + kVec <= V) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + e0));
        const T* t = reinterpret_cast<const T*>(&w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = to_float(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = e0 + i >= 0 && e0 + i < V ? to_float(row[e0 + i]) : 0.0f;
    }
    uint32_t worst = 0;  // as bits, what is negative, infinite or NaN is above every other
#pragma unroll
    for (int i = 0; i < kVec; ++i) worst = max(worst, __float_as_uint(x[i]));
    if (worst >= 0x7f800000u) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = clean(x[i], bad);
    }
}

template <typename T, bool kDrafter>
__global__ void __cluster_dims__(kCtasV, 1, 1) __launch_bounds__(kThreadsV) draft_verify_kernel(const VerifyArgs a) {
    constexpr int kVec = Row<T>::kVec;
    extern __shared__ uint32_t gone[];  // without a drafter: a bit for each token of the CTA's slice that was rejected
    __shared__ int node_parent[kNodes], node_token[kNodes];
    __shared__ float node_coin[kNodes], node_p[kNodes], node_q[kNodes];
    __shared__ double warp_sum[kWarpsV];
    __shared__ double cta_sum[2];  // of this pass and the last one, which another CTA may still read
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster.block_rank();
    const int b = blockIdx.x / kCtasV;
    pdl_wait();
    pdl_launch_dependents();
    const int32_t c0 = a.cu_seqlens_q[b], c1 = a.cu_seqlens_q[b + 1], n = c1 - c0;
    const bool fine = c0 >= 0 && c1 >= c0 && c1 <= a.T && n <= a.max_q_len;
    int32_t* path = a.path + (int64_t)b * a.max_path;
    int32_t* out = a.out_tokens + (int64_t)b * a.max_path;
    if (!fine || n == 0) {  // the same for the cluster
        if (rank == 0) {
            for (int i = tid; i < a.max_path; i += kThreadsV) path[i] = out[i] = -1;
            if (tid == 0) {
                a.n_path[b] = 0;
                if (!fine) report(a.dev_status, IDX_STATUS_BAD_LEN);
            }
        }
        return;
    }

    const T* target = static_cast<const T*>(a.target) + (int64_t)c0 * a.target_stride;
    const T* draft = kDrafter ? static_cast<const T*>(a.draft) + (int64_t)c0 * a.draft_stride : nullptr;
    const int V = a.V;
    bool bad = false, bad_token = false;

    // Nodes from .. from + kNodes - 1, each with what its parent's rows say of its token. Values of nodes that are never
    // tested are not judged.
    auto stage = [&](int from) {
        __syncthreads();
        const int j = from + tid;
        if (j < n) {
            const int up = a.parents[c0 + j], x = a.tokens[c0 + j];
            node_parent[tid] = up;
            node_token[tid] = x;
            node_coin[tid] = a.coins[c0 + j];
            if (up >= 0 && up < j && x >= 0 && x < V) {
                node_p[tid] = to_float(target[(int64_t)up * a.target_stride + x]);
                if constexpr (kDrafter) node_q[tid] = to_float(draft[(int64_t)up * a.draft_stride + x]);
            }
        }
        __syncthreads();
        return from;
    };

    // ---- a pass: the sums of what is left of the row of node `cur` ----------------------------------------------
    int cur = 0, pass = 0, from = 0;
    const T* p = target;
    const T* q = draft;
    // the vectors of the row, this CTA's and this warp's
    int off = 0, k0 = 0, k1 = 0, e_first = 0;
    bool q_whole = false;
    auto place = [&]() {
        p = target + (int64_t)cur * a.target_stride;
        off = Row<T>{p}.off();
        if constexpr (kDrafter) {
            q = draft + (int64_t)cur * a.draft_stride;
            q_whole = Row<T>{q}.off() == off;
        }
        const int all = (V + off + kVec - 1) / kVec, slice = (all + kCtasV - 1) / kCtasV;
        const int s0 = min(rank * slice, all), s1 = min(s0 + slice, all), part = (s1 - s0 + kWarpsV - 1) / kWarpsV;
        k0 = min(s0 + warp * part, s1);
        k1 = min(k0 + part, s1);
        e_first = s0 * kVec - off;  // of the CTA
    };
    // weights of vector k: p, without the rejected tokens (mask) or less cut times q (c_hi + c_lo)
    auto weights = [&](int k, int how, float c_hi, float c_lo, Pair (&w)[kVec]) {
        const int e0 = k * kVec - off;
        float x[kVec];
        load<T>(p, e0, V, true, bad, x);
        if (kDrafter && how) {
            float y[kVec];
            load<T>(q, e0, V, q_whole, bad, y);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float t = __fmul_rn(c_hi, y[i]), te = __fmaf_rn(c_lo, y[i], __fmaf_rn(c_hi, y[i], -t));
                const float d = __fsub_rn(x[i], t), z = __fsub_rn(d, x[i]);
                const float e = __fsub_rn(__fsub_rn(__fsub_rn(x[i], __fsub_rn(d, z)), __fadd_rn(t, z)), te);
                const bool some = __fadd_rn(d, e) > 0.0f;
                w[i] = Pair{some ? d : 0.0f, some ? e : 0.0f};
            }
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                if (!kDrafter && how) {
                    const int v = max(e0 + i, 0) - max(e_first, 0);
                    if (e0 + i >= 0 && e0 + i < V && (gone[v >> 5] >> (v & 31)) & 1u) x[i] = 0.0f;
                }
                w[i] = Pair{x[i], 0.0f};
            }
        }
    };
    double before_cta = 0.0;  // sums of the slices in front of this CTA's
    auto total = [&](int how, double cut) -> double {
        const float c_hi = (float)cut, c_lo = (float)(cut - (double)c_hi);
        Pair s[4] = {};
#pragma unroll 4
        for (int k = k0 + lane; k < k1; k += 32) {
            Pair w[kVec];
            weights(k, how, c_hi, c_lo, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) add(s[i & 3], w[i]);
        }
        add(s[0], s[1]);
        add(s[2], s[3]);
        add(s[0], s[2]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Pair y{__shfl_xor_sync(kFull, s[0].hi, o), __shfl_xor_sync(kFull, s[0].lo, o)};
            add(s[0], y);
        }
        __syncthreads();  // warp_sum has been read
        if (lane == 0) warp_sum[warp] = (double)s[0].hi + (double)s[0].lo;
        __syncthreads();
        if (tid == 0) {
            double t = 0.0;
            for (int w = 0; w < kWarpsV; ++w) t += warp_sum[w];
            cta_sum[pass & 1] = t;
        }
        cluster.sync();
        double t = 0.0;
        for (int c = 0; c < kCtasV; ++c) {
            if (c == rank) before_cta = t;
            t += *cluster.map_shared_rank(&cta_sum[pass & 1], c);
        }
        ++pass;
        return t;
    };

    // ---- the walk -----------------------------------------------------------------------------------------------
    int length = 1, rejected = 0;
    double cut = 0.0, mass = 1.0;
    const bool writes = rank == 0 && tid == 0;
    if (writes) path[0] = 0;
    from = stage(0);
    for (int j = 1; length < a.max_path && j < n;) {
        if (j >= from + kNodes) from = stage(j);
        // the next child, found by each warp for itself
        const int end = min(n, from + kNodes);
        int child = -1;
        for (; j < end; j += 32) {
            const unsigned hit = __ballot_sync(kFull, j + lane < end && node_parent[j + lane - from] == cur);
            if (hit) {
                child = j + __ffs(hit) - 1;
                break;
            }
        }
        if (child < 0) {
            j = end;
            continue;
        }
        j = child + 1;
        const int x = node_token[child - from];
        if (x < 0 || x >= V) {
            bad_token = true;
            continue;
        }
        const double u = node_coin[child - from];
        double px = clean(node_p[child - from], bad);
        bool yes;
        if constexpr (kDrafter) {
            const double qx = clean(node_q[child - from], bad);
            yes = __dmul_rn(__dmul_rn(u, qx), mass) < __dsub_rn(px, __dmul_rn(cut, qx));
            if (!yes) {
                if (!rejected) place();
                cut += mass;
                mass = total(1, cut);
            }
        } else {
            // rejected here before: an earlier child with this token
            for (int i = cur + 1; rejected && i < child; i += 32) {
                const bool same = i + lane < child && a.parents[c0 + i + lane] == cur && a.tokens[c0 + i + lane] == x;
                if (__any_sync(kFull, same)) {
                    px = 0.0;
                    break;
                }
            }
            yes = __dmul_rn(u, mass) < px;
            if (!yes) mass = mass > px ? mass - px : 0.0;
        }
        if (!yes) {
            ++rejected;
            continue;
        }
        if (writes) {
            path[length] = child;
            out[length - 1] = x;
        }
        ++length;
        cur = child;
        cut = 0.0;
        mass = 1.0;
        rejected = 0;
    }

    // ---- the draw -----------------------------------------------------------------------------------------------
    int how = rejected ? 1 : 0;
    double all = mass;
    if (!kDrafter || !rejected) {
        place();
        if (!kDrafter && rejected) {
            const int v0 = max(e_first, 0), slice = ((V + off + kVec - 1) / kVec + kCtasV - 1) / kCtasV * kVec;
            for (int i = tid; i < (slice + 31) / 32; i += kThreadsV) gone[i] = 0;
            __syncthreads();
            for (int i = cur + 1 + tid; i < n; i += kThreadsV) {
                const int x = a.tokens[c0 + i], v = x - v0;
                if (a.parents[c0 + i] == cur && x >= 0 && x < V && v >= 0 && v < slice) atomicOr(&gone[v >> 5], 1u << (v & 31));
            }
            __syncthreads();
        }
        all = total(how, cut);
    }
    if (!(all > 0.0)) {  // nothing is left of p: p itself
        how = 0;
        all = total(0, 0.0);
    }
    float r = a.last[b];
    const bool bad_coin = !(r >= 0.0f && r < 1.0f);
    if (!(r >= 0.0f)) r = 0.0f;
    const double goal = __dmul_rn((double)r, all);
    // the CTA, and in it the warp, whose part holds the border; with r >= 1 the last that holds anything
    int owner = 0;
    {
        double t = 0.0;
        for (int c = 0; c < kCtasV; ++c) {
            const double x = *cluster.map_shared_rank(&cta_sum[(pass - 1) & 1], c);
            if (x > 0.0) owner = c;
            t += x;
            if (t > goal) break;
        }
    }
    if (rank == owner) {
        int at = 0;
        double before = before_cta, t = before_cta;
        for (int w = 0; w < kWarpsV; ++w) {
            if (warp_sum[w] > 0.0) {
                at = w;
                before = t;
            }
            t += warp_sum[w];
            if (t > goal) break;
        }
        if (warp == at) {
            const float c_hi = (float)cut, c_lo = (float)(cut - (double)c_hi);
            int found = -1;
            for (int k = k0; k < k1; k += 32) {
                Pair w[kVec];
                double x = 0.0;
                int last = -1;  // this lane's last element that weighs anything
                if (k + lane < k1) {
                    weights(k + lane, how, c_hi, c_lo, w);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
                        x += (double)w[i].hi + (double)w[i].lo;
                        if (__fadd_rn(w[i].hi, w[i].lo) > 0.0f) last = i;
                    }
                }
                double upto = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(kFull, upto, o);
                    if (lane >= o) upto += y;
                }
                const unsigned passes = __ballot_sync(kFull, last >= 0 && before + upto > goal);
                const unsigned some = __ballot_sync(kFull, last >= 0);
                if (!passes) {
                    if (some) found = (k + 31 - __clz(some)) * kVec - off + __shfl_sync(kFull, last, 31 - __clz(some));
                    before += __shfl_sync(kFull, upto, 31);
                    continue;
                }
                const int l = __ffs(passes) - 1;
                if (lane == l) {
                    double t2 = before + (upto - x);
                    int hit = last;
#pragma unroll
                    for (int i = kVec - 1; i >= 0; --i) {
                        double s = t2;
                        for (int m = 0; m <= i; ++m) s += (double)w[m].hi + (double)w[m].lo;
                        if (__fadd_rn(w[i].hi, w[i].lo) > 0.0f && s > goal) hit = i;
                    }
                    found = (k + l) * kVec - off + hit;
                }
                found = __shfl_sync(kFull, found, l);
                break;
            }
            if (lane == 0) {
                out[length - 1] = found;
                a.n_path[b] = length;
                if (found < 0 || bad_coin || bad_token) report(a.dev_status, IDX_STATUS_BAD_VALUE);
            }
        }
    }
    if (rank == 0) {
        for (int i = length + tid; i < a.max_path; i += kThreadsV) path[i] = out[i] = -1;
    }
    if (bad) report(a.dev_status, IDX_STATUS_BAD_VALUE);
    cluster.sync();  // nobody reads another CTA's sums any more
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)a.B * kCtasV), block(kThreadsV);
    if (a.draft) return launch_pdl(draft_verify_kernel<T, true>, grid, block, 0, st, a);
    const int vec = 16 / (int)sizeof(T);
    const int slice = (((a.V + 2 * vec - 2) / vec + kCtasV - 1) / kCtasV) * vec;  // as if no row were aligned
    return launch_pdl(draft_verify_kernel<T, false>, grid, block, (size_t)(slice + 31) / 32 * 4, st, a);
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyArgs& a, cudaStream_t st) {
    if (a.ptype == IDX_FP32) return launch<float>(a, st);
    return a.ptype == IDX_BF16 ? launch<__nv_bfloat16>(a, st) : launch<__half>(a, st);
}

}  // namespace idx
