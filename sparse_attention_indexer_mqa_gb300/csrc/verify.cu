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
// would move one draw in a hundred. fp64 has a 64th of fp32's rate here (a few scalar operations of it in every warp
// were most of a small call's time), so weights, sums and what is compared with them are pairs of fp32: a value and what its
// rounding lost, by error-free sums and products, about 2^-46 of the sum. Two elements go through one packed instruction.
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
constexpr int kAhead = 2;          // vectors of either row that a thread has in flight

// A value and what its roundings lost: hi + lo.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ void add(Pair& s, float x) {  // s.hi + x exactly, as a sum and its error
    const float t = __fadd_rn(s.hi, x), b = __fsub_rn(t, s.hi);
    s.lo = __fadd_rn(s.lo, __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s.hi = t;
}
__device__ __forceinline__ void add(Pair& s, const Pair& x) {
    add(s, x.hi);
    s.lo = __fadd_rn(s.lo, x.lo);
}
__device__ __forceinline__ Pair tidy(const Pair& x) {  // hi the nearest fp32 of the whole
    const float t = __fadd_rn(x.hi, x.lo);
    return Pair{t, __fsub_rn(x.lo, __fsub_rn(t, x.hi))};
}
__device__ __forceinline__ Pair times(const Pair& x, float y) {
    const float t = __fmul_rn(x.hi, y);
    return Pair{t, __fmaf_rn(x.lo, y, __fmaf_rn(x.hi, y, -t))};
}
__device__ __forceinline__ Pair less(const Pair& x, const Pair& y) {  // x - y
    Pair d = x;
    add(d, Pair{-y.hi, -y.lo});
    return d;
}
__device__ __forceinline__ bool positive(const Pair& x) { return __fadd_rn(x.hi, x.lo) > 0.0f; }

// The sum of lanes 0 .. n - 1's, the same in every lane (each lane's own would differ in the last bits).
template <int n>
__device__ __forceinline__ Pair lane0_sum(Pair x) {
#pragma unroll
    for (int o = n / 2; o > 0; o >>= 1) {
        const Pair y{__shfl_down_sync(kFull, x.hi, o), __shfl_down_sync(kFull, x.lo, o)};
        add(x, y);
    }
    return Pair{__shfl_sync(kFull, x.hi, 0), __shfl_sync(kFull, x.lo, 0)};
}
__device__ __forceinline__ Pair running_sum(Pair x) {  // of lanes 0 .. this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y{__shfl_up_sync(kFull, x.hi, o), __shfl_up_sync(kFull, x.lo, o)};
        if ((threadIdx.x & 31) >= o) add(x, y);
    }
    return x;
}

// Lane i holds the sum of part i. The first part behind whose end the running sum is past the goal, or else the last that
// holds anything (0 if none does); the goal loses what lies in front of that part. The same in every lane.
__device__ __forceinline__ int first_past(const Pair& x, Pair& goal) {
    const Pair upto = running_sum(x);
    const unsigned some = __ballot_sync(kFull, positive(x));
    const unsigned past = __ballot_sync(kFull, positive(x) && positive(less(upto, goal)));
    const int part = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
    const Pair front{__shfl_sync(kFull, upto.hi, max(part - 1, 0)), __shfl_sync(kFull, upto.lo, max(part - 1, 0))};
    if (part) goal = less(goal, front);
    return part;
}

// Two values in one instruction, each rounded as by itself.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
        " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
        " mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }

// Two pairs.
struct Pair2 {
    float2 hi, lo;
};
__device__ __forceinline__ void add(Pair2& s, const Pair2& x) {
    const float2 t = add2(s.hi, x.hi), b = sub2(t, s.hi);
    s.lo = add2(s.lo, add2(add2(sub2(s.hi, sub2(t, b)), sub2(x.hi, b)), x.lo));
    s.hi = t;
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

// Element by element, for a vector that the row's end cuts or that lies on no 16-byte boundary.
template <typename T>
__device__ __forceinline__ uint4 gather(const T* row, int e0, int V) {
    constexpr int kVec = 16 / sizeof(T);
    uint4 w = make_uint4(0, 0, 0, 0);
    T* t = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (e0 + i >= 0 && e0 + i < V) t[i] = row[e0 + i];
    return w;
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, bool& bad, float (&x)[16 / sizeof(T)]) {
    constexpr int kVec = 16 / sizeof(T);
    const T* t = reinterpret_cast<const T*>(&w);
    uint32_t worst = 0;  // as bits, what is negative, infinite or NaN is above every other
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        x[i] = to_float(t[i]);
        worst = max(worst, __float_as_uint(x[i]));
    }
    if (worst >= 0x7f800000u) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = clean(x[i], bad);
    }
}

template <typename T, bool kDrafter>
__global__ void __cluster_dims__(kCtasV, 1, 1) __launch_bounds__(kThreadsV, 4) draft_verify_kernel(const VerifyArgs a) {
    constexpr int kVec = Row<T>::kVec;
    extern __shared__ uint32_t gone[];  // without a drafter: a bit for each token of the CTA's slice that was rejected
    __shared__ int node_parent[kNodes], node_token[kNodes];
    __shared__ float node_coin[kNodes], node_p[kNodes], node_q[kNodes];
    __shared__ Pair warp_sum[kWarpsV];
    __shared__ Pair cta_sum[2];  // of this pass and the last one, which another CTA may still read
    __shared__ int first_thread, last_thread;
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
    // the row's vectors: this CTA's slice, a warp's part of it
    int off = 0, s0 = 0, s1 = 0, k0 = 0, k1 = 0;
    bool q_whole = false;
    auto part_of = [&](int w) {
        const int part = (s1 - s0 + kWarpsV - 1) / kWarpsV;
        k0 = min(s0 + w * part, s1);
        k1 = min(k0 + part, s1);
    };
    auto place = [&]() {
        p = target + (int64_t)cur * a.target_stride;
        off = Row<T>{p}.off();
        if constexpr (kDrafter) {
            q = draft + (int64_t)cur * a.draft_stride;
            q_whole = Row<T>{q}.off() == off;
        }
        const int all = (V + off + kVec - 1) / kVec, slice = (all + kCtasV - 1) / kCtasV;
        s0 = min(rank * slice, all);
        s1 = min(s0 + slice, all);
        part_of(warp);
    };
    // Vector k of either row, as it is in memory. Only a row's first and last vector may be cut by its ends.
    auto cut_short = [&](int k) { return k * kVec < off || (k + 1) * kVec - off > V; };
    auto fetch = [&](int k, int how, uint4& x, uint4& y) {
        const int e0 = k * kVec - off;
        const bool cut_off = cut_short(k);
        x = y = make_uint4(0, 0, 0, 0);
        if (!cut_off) x = __ldg(reinterpret_cast<const uint4*>(p + e0));
        if (kDrafter && how && !cut_off && q_whole) y = __ldg(reinterpret_cast<const uint4*>(q + e0));
    };
    auto fetch_rest = [&](int k, int how, uint4& x, uint4& y) {
        const bool cut_off = cut_short(k);
        if (cut_off) x = gather(p, k * kVec - off, V);
        if (kDrafter && how && (cut_off || !q_whole)) y = gather(q, k * kVec - off, V);
    };
    // its weights, two to a Pair2: p, without the rejected tokens or less cut times q
    auto weights = [&](int k, int how, const Pair& cut, const uint4& px, const uint4& qx, Pair2 (&w)[kVec / 2]) {
        const int e0 = k * kVec - off;
        float x[kVec];
        unpack<T>(px, bad, x);
        if (kDrafter && how) {
            float y[kVec];
            unpack<T>(qx, bad, y);
            const float2 c = make_float2(cut.hi, cut.hi), c_lo = make_float2(cut.lo, cut.lo), nc = make_float2(-cut.hi, -cut.hi);
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
                const float2 x2 = make_float2(x[2 * i], x[2 * i + 1]), y2 = make_float2(y[2 * i], y[2 * i + 1]);
                const float2 nt = mul2(nc, y2), te = fma2(c_lo, y2, fma2(c, y2, nt));  // cut * y = te - nt
                const float2 d = add2(x2, nt), z = sub2(d, x2);
                const float2 e = sub2(add2(sub2(x2, sub2(d, z)), sub2(nt, z)), te);
                const float2 s = add2(d, e);
                w[i].hi = make_float2(s.x > 0.0f ? d.x : 0.0f, s.y > 0.0f ? d.y : 0.0f);
                w[i].lo = make_float2(s.x > 0.0f ? e.x : 0.0f, s.y > 0.0f ? e.y : 0.0f);
            }
        } else {
            if (!kDrafter && how) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const int v = e0 + i - max(s0 * kVec - off, 0);
                    if (e0 + i >= 0 && e0 + i < V && (gone[v >> 5] >> (v & 31)) & 1u) x[i] = 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) w[i] = Pair2{make_float2(x[2 * i], x[2 * i + 1]), make_float2(0.0f, 0.0f)};
        }
    };
    auto total = [&](int how, const Pair& cut) -> Pair {
        Pair2 s[2] = {};
        for (int k = k0 + lane; k < k1; k += 32 * kAhead) {
            uint4 x[kAhead], y[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {  // past the part's end its last vector again, which is not counted
                fetch(min(k + 32 * u, k1 - 1), how, x[u], y[u]);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (k + 32 * u >= k1) break;
                fetch_rest(k + 32 * u, how, x[u], y[u]);
                Pair2 w[kVec / 2];
                weights(k + 32 * u, how, cut, x[u], y[u], w);
#pragma unroll
                for (int i = 0; i < kVec / 2; ++i) add(s[i & 1], w[i]);
            }
        }
        add(s[0], s[1]);
        Pair mine{s[0].hi.x, s[0].lo.x};
        add(mine, Pair{s[0].hi.y, s[0].lo.y});
        mine = lane0_sum<32>(mine);
        __syncthreads();  // warp_sum has been read
        if (lane == 0) warp_sum[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const Pair x = lane0_sum<kWarpsV>(warp_sum[lane % kWarpsV]);
            if (lane == 0) cta_sum[pass & 1] = x;
        }
        cluster.sync();
        const Pair x = lane0_sum<kCtasV>(*cluster.map_shared_rank(&cta_sum[pass & 1], lane % kCtasV));
        ++pass;
        return tidy(x);
    };

    // ---- the walk -----------------------------------------------------------------------------------------------
    int length = 1, rejected = 0;
    const Pair zero{0.0f, 0.0f}, one{1.0f, 0.0f};
    Pair cut = zero, mass = one;
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
        const float u = node_coin[child - from];
        float px = clean(node_p[child - from], bad);
        bool yes;
        if constexpr (kDrafter) {
            const float qx = clean(node_q[child - from], bad);
            // u q S < p - c q; a coin that is no number rejects
            const float uq = __fmul_rn(u, qx);
            Pair need = times(mass, uq);
            add(need, __fmul_rn(mass.hi, __fmaf_rn(u, qx, -uq)));
            yes = positive(less(less(Pair{px, 0.0f}, times(cut, qx)), need));
            if (!yes) {
                if (!rejected) place();
                add(cut, mass);
                cut = tidy(cut);
                mass = total(1, cut);
            }
        } else {
            // rejected here before: an earlier child with this token
            for (int i = cur + 1; rejected && i < child; i += 32) {
                const bool same = i + lane < child && a.parents[c0 + i + lane] == cur && a.tokens[c0 + i + lane] == x;
                if (__any_sync(kFull, same)) {
                    px = 0.0f;
                    break;
                }
            }
            yes = positive(less(Pair{px, 0.0f}, times(mass, u)));
            if (!yes) {
                add(mass, -px);
                mass = positive(mass) ? tidy(mass) : zero;
            }
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
        cut = zero;
        mass = one;
        rejected = 0;
    }

    // ---- the draw -----------------------------------------------------------------------------------------------
    int how = rejected ? 1 : 0;
    Pair all = mass;
    if (!kDrafter || !rejected) {
        place();
        if (!kDrafter && rejected) {
            const int v0 = max(s0 * kVec - off, 0), slice = ((V + off + kVec - 1) / kVec + kCtasV - 1) / kCtasV * kVec;
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
    if (!positive(all)) {  // nothing is left of p: p itself
        how = 0;
        all = total(0, zero);
    }
    float r = a.last[b];
    const bool bad_coin = !(r >= 0.0f && r < 1.0f);
    if (!(r >= 0.0f)) r = 0.0f;
    Pair goal = times(all, r);  // passed by a sum that is above it
    // The border: the CTA's slice that holds it, the warp's part in that, a thread's piece of that, the element. Where
    // rounding or r >= 1 puts the goal behind everything, the last one that weighs anything.
    const int owner = first_past(lane < kCtasV ? *cluster.map_shared_rank(&cta_sum[(pass - 1) & 1], lane % kCtasV) : zero, goal);
    if (rank == owner) {
        part_of(first_past(lane < kWarpsV ? warp_sum[lane % kWarpsV] : zero, goal));
        const int piece = (k1 - k0 + kThreadsV - 1) / kThreadsV, a0 = min(k0 + tid * piece, k1), a1 = min(a0 + piece, k1);
        auto vector = [&](int k, Pair2 (&x)[kVec / 2]) {
            uint4 px, qx;
            fetch(k, how, px, qx);
            fetch_rest(k, how, px, qx);
            weights(k, how, cut, px, qx, x);
        };
        Pair s = zero;
        for (int k = a0; k < a1; ++k) {
            Pair2 x[kVec / 2];
            vector(k, x);
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
                add(s, Pair{x[i].hi.x, x[i].lo.x});
                add(s, Pair{x[i].hi.y, x[i].lo.y});
            }
        }
        const Pair upto = running_sum(s);
        __syncthreads();  // every warp has read warp_sum
        if (lane == 31) warp_sum[warp] = upto;
        if (tid == 0) {
            first_thread = kThreadsV;
            last_thread = -1;
        }
        __syncthreads();
        for (int x = 0; x < warp; ++x) goal = less(goal, warp_sum[x]);
        const unsigned some = __ballot_sync(kFull, positive(s));
        const unsigned past = __ballot_sync(kFull, positive(s) && positive(less(upto, goal)));
        if (lane == 0) {
            if (past) atomicMin(&first_thread, warp * 32 + __ffs(past) - 1);
            if (some) atomicMax(&last_thread, warp * 32 + 31 - __clz(some));
        }
        __syncthreads();
        const int mine = first_thread < kThreadsV ? first_thread : max(last_thread, 0);
        if (tid == mine) {
            int found = -1;
            bool done = false;
            Pair t = less(upto, s);
            for (int k = a0; k < a1 && !done; ++k) {
                Pair2 x[kVec / 2];
                vector(k, x);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const Pair w = i & 1 ? Pair{x[i / 2].hi.y, x[i / 2].lo.y} : Pair{x[i / 2].hi.x, x[i / 2].lo.x};
                    add(t, w);
                    if (!done && positive(w)) {
                        found = k * kVec - off + i;
                        done = positive(less(t, goal));
                    }
                }
            }
            out[length - 1] = found;
            a.n_path[b] = length;
            if (found < 0 || bad_coin || bad_token) report(a.dev_status, IDX_STATUS_BAD_VALUE);
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
