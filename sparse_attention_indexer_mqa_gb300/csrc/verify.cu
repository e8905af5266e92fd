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
// could move up to one draw in a hundred. fp64 has a 64th of fp32's rate here, so weights, sums and what is compared with them
// are pairs of fp32: a value and what its rounding lost, by error-free sums and products, about 2^-46 of the sum.
//
// A cluster of up to eight CTAs per request: the row is cut into a slice for each, a slice into the CTA's warps' parts. All
// threads follow the walk by themselves; a pass ends with one cluster barrier, behind which every CTA adds up the
// slices' sums in the same order. What the walk asks of each node (its parent, token, number and the two
// probabilities) is fetched for 256 nodes at once, so that a step between passes is no chain of loads. The CTA whose slice holds
// the draw's border searches the part of the warp that holds it with all its threads.
//
// Measured. 64 trees of 32 nodes, 131072 tokens, fp32: 28.1 us in a replayed graph, whose rows (67 MB) stay in L2; 34 among
// other calls, 40 with L2 flushed and events included. One pass for each is 9.9 us at the copy rate, but a request of three or
// four passes, each behind the decision that the one before allows, sets the end; a pass of few requests is bound by the
// loads' latency, four vectors of either row a thread, and the barriers. One chain of 4 drafts,
// 49999 tokens, bf16: 7.9 us in a graph: launch, three dependent loads, the pass with its barriers, the search; a call from the
// host takes 10. Before: a CTA per request, sums in fp64 907; a cluster 68; batched loads and the search
// by a whole CTA 53; no fp64 36; no test per vector 30. 16-bit probabilities take as long (bf16 28.8, fp16 27.3): passes in turn, not
// bytes. Rows that begin at other places within 16 bytes for the two sides (a padded vocabulary on one side) have q's entries
// fetched one by one: 68 us for those 64 trees in fp32, 60 in bf16; a chain of 4 drafts, 50000 tokens, 15.2 against 10.2. An odd
// vocabulary, rows of every alignment but alike on both sides: 37 in fp32, 40 in bf16.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace idx {

namespace {

constexpr int kThreadsV = 256, kWarpsV = kThreadsV / 32, kCtasMost = 8;
constexpr int kNodes = kThreadsV;  // nodes that are staged at once
constexpr int kAhead = 4;          // vectors of either row that a thread has on their way

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
template <int n = 32>
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

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// What is no probability (negative, NaN, infinite) counts as zero.
__device__ __forceinline__ float clean(float x, bool& bad) {
    const bool ok = x >= 0.0f && x < __int_as_float(0x7f800000);
    bad |= !ok;
    return ok ? x : 0.0f;
}
// A vector with such an entry: a call, for it is rare and its code would be fetched by every small call.
template <typename T>
__device__ __noinline__ uint4 clean_vector(uint4 w, int32_t* status) {
    constexpr int kVec = 16 / sizeof(T);
    T* t = reinterpret_cast<T*>(&w);
    bool bad = false;
    for (int i = 0; i < kVec; ++i)
        if (!(clean(to_float(t[i]), bad) > 0.0f)) t[i] = T(0.0f);
    if (bad) report(status, IDX_STATUS_BAD_VALUE);
    return w;
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
__device__ __noinline__ uint4 gather(const T* row, int e0, int V) {
    constexpr int kVec = 16 / sizeof(T);
    uint4 w = make_uint4(0, 0, 0, 0);
    T* t = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (e0 + i >= 0 && e0 + i < V) t[i] = row[e0 + i];
    return w;
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[16 / sizeof(T)]) {
#pragma unroll
    for (int i = 0; i < 16 / (int)sizeof(T); ++i) x[i] = to_float(reinterpret_cast<const T*>(&w)[i]);
}

// How a pass weighs an entry: p as it is, p less q (a node's first pass, the only one of most), p less cut times q,
// p without the rejected tokens.
enum { kAll, kLessQ, kLessCutQ, kWithout };

// The weights of a vector's entries, which have to be probabilities; gone: a bit for each that was rejected.
template <int kHow, int kVec>
__device__ __forceinline__ void weigh(const Pair& cut, uint32_t gone, const float (&x)[kVec], const float (&y)[kVec], Pair (&w)[kVec]) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if constexpr (kHow == kLessQ) {  // held to x, q leaves no negative difference, and its error takes two operations
            const float t = fminf(y[i], x[i]), d = __fsub_rn(x[i], t);
            w[i] = Pair{d, __fsub_rn(__fsub_rn(x[i], d), t)};
        } else if constexpr (kHow == kLessCutQ) {  // so does this one's where x is larger or nearly so; elsewhere it weighs nothing
            const float c = __fmul_rn(cut.hi, y[i]), ce = __fmaf_rn(cut.lo, y[i], __fmaf_rn(cut.hi, y[i], -c));
            const float d = __fsub_rn(x[i], c), e = __fsub_rn(__fsub_rn(__fsub_rn(x[i], d), c), ce);
            const bool some = __fadd_rn(d, e) > 0.0f;
            w[i] = Pair{some ? d : 0.0f, some ? e : 0.0f};
        } else {
            w[i] = Pair{kHow == kWithout && (gone >> i) & 1u ? 0.0f : x[i], 0.0f};
        }
    }
}

template <typename T, bool kDrafter>
__global__ void __launch_bounds__(kThreadsV, 4) draft_verify_kernel(const VerifyArgs a) {
    constexpr int kVec = Row<T>::kVec;
    // without a drafter: a bit for each token of the CTA's slice that was rejected, from the slice's first vector on
    extern __shared__ uint32_t gone[];
    __shared__ int node_parent[kNodes], node_token[kNodes];
    __shared__ float node_coin[kNodes], node_p[kNodes], node_q[kNodes];
    __shared__ Pair warp_sum[kWarpsV];
    __shared__ Pair cta_sum[2];  // of this pass and the last one, which another CTA may still read
    __shared__ int first_thread, last_thread;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), b = blockIdx.x / ctas;
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
    const Pair zero{0.0f, 0.0f}, one{1.0f, 0.0f};
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
        const int all = (V + off + kVec - 1) / kVec, slice = (all + ctas - 1) / ctas;
        s0 = min(rank * slice, all);
        s1 = min(s0 + slice, all);
        part_of(warp);
    };
    // Vector k of either row, as it is in memory; only a row's first and last one may be cut by its ends.
    auto cut_short = [&](int k) { return k * kVec < off || (k + 1) * kVec - off > V; };
    auto fetch_p = [&](int k) -> uint4 {
        const int e0 = k * kVec - off;
        return cut_short(k) ? gather(p, e0, V) : __ldg(reinterpret_cast<const uint4*>(p + e0));
    };
    auto fetch_q = [&](int k) -> uint4 {
        const int e0 = k * kVec - off;
        return cut_short(k) || !q_whole ? gather(q, e0, V) : __ldg(reinterpret_cast<const uint4*>(q + e0));
    };
    auto gone_bits = [&](int k) -> uint32_t { return gone[((k - s0) * kVec) >> 5] >> (((k - s0) * kVec) & 31); };
    // The weights of a vector of any kind, its entries looked at one by one.
    auto careful = [&](int how, int k, const Pair& cut, Pair (&w)[kVec]) {
        float x[kVec], y[kVec];
        unpack<T>(clean_vector<T>(fetch_p(k), a.dev_status), x);
        if (how == kAll) {
            weigh<kAll, kVec>(cut, 0, x, x, w);
        } else if constexpr (kDrafter) {
            unpack<T>(clean_vector<T>(fetch_q(k), a.dev_status), y);
            weigh<kLessCutQ, kVec>(cut, 0, x, y, w);
        } else {
            weigh<kWithout, kVec>(cut, gone_bits(k), x, x, w);
        }
    };
    auto total = [&](int how, const Pair& cut) -> Pair {
        Pair s[4] = {};
        const bool with_q = kDrafter && how != kAll;
        // Vectors that lie whole in the row, four of each row on their way at once and no test but the loop's: what an
        // entry's bits are is asked behind it. As bits, what is negative, infinite or NaN is above every other entry; all
        // entries' bits together are so too, and are else only where one is 2 or more, which is then looked at in vain.
        const int f0 = max(k0, off > 0), f1 = with_q && !q_whole ? f0 : max(f0, min(k1, (V + off) / kVec));
        const uint4* pv = reinterpret_cast<const uint4*>(p - off);
        const uint4* qv = kDrafter ? reinterpret_cast<const uint4*>(q - off) : nullptr;
        uint32_t bits = 0;
        auto fast = [&](auto tag) {
            constexpr int kHow = decltype(tag)::value;
            constexpr bool kQ = kHow == kLessQ || kHow == kLessCutQ;
            auto take = [&](int k, const uint4& px, const uint4& qx) {
                float x[kVec], y[kVec];
                unpack<T>(px, x);
                unpack<T>(qx, y);
#pragma unroll
                for (int i = 0; i < kVec; ++i) bits |= __float_as_uint(x[i]) | (kQ ? __float_as_uint(y[i]) : 0);
                Pair w[kVec];
                weigh<kHow, kVec>(cut, kHow == kWithout ? gone_bits(k) : 0, x, y, w);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    if constexpr (kQ)
                        add(s[i & 3], w[i]);
                    else
                        add(s[i & 3], w[i].hi);
                }
            };
            int k = f0 + lane;
#pragma unroll 1
            for (; k + 32 * (kAhead - 1) < f1; k += 32 * kAhead) {
                uint4 px[kAhead], qx[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    px[u] = __ldg(pv + k + 32 * u);
                    if constexpr (kQ) qx[u] = __ldg(qv + k + 32 * u);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) take(k + 32 * u, px[u], kQ ? qx[u] : px[u]);
            }
#pragma unroll 1
            for (; k < f1; k += 32) {
                const uint4 px = __ldg(pv + k);
                take(k, px, kQ ? __ldg(qv + k) : px);
            }
        };
        if (how == kAll)
            fast(std::integral_constant<int, kAll>{});
        else if constexpr (!kDrafter)
            fast(std::integral_constant<int, kWithout>{});
        else if (how == kLessQ)
            fast(std::integral_constant<int, kLessQ>{});
        else
            fast(std::integral_constant<int, kLessCutQ>{});
        const bool again = bits >= 0x7f800000u;  // this thread's once more
        if (again) s[0] = s[1] = s[2] = s[3] = zero;
        // What the row's ends cut, or all of it where p and q are not aligned alike, and once more what this thread has thrown
        // away: a vector from f0 on is the same thread's as above; the only one that can lie in front of f0 is k0.
#pragma unroll 1
        for (int k = k0 < f0 && lane == 31 ? k0 : f0 + lane; k < k1; k += 32) {
            if (!again && k >= f0 && k < f1) {
                k += (f1 - 1 - k) / 32 * 32;
                continue;
            }
            Pair w[kVec];
            careful(how, k, cut, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) add(s[i & 3], w[i]);
        }
        add(s[0], s[1]);
        add(s[2], s[3]);
        add(s[0], s[2]);
        s[0] = lane0_sum(s[0]);
        __syncthreads();  // warp_sum has been read
        if (lane == 0) warp_sum[warp] = s[0];
        __syncthreads();
        if (warp == 0) {
            const Pair x = lane0_sum<kWarpsV>(warp_sum[lane % kWarpsV]);
            if (lane == 0) cta_sum[pass & 1] = x;
        }
        cluster.sync();
        const Pair x = lane0_sum<kCtasMost>(lane < ctas ? *cluster.map_shared_rank(&cta_sum[pass & 1], lane) : zero);
        ++pass;
        return tidy(x);
    };

    // ---- the walk -----------------------------------------------------------------------------------------------
    int length = 1, rejected = 0;
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
                mass = total(rejected ? kLessCutQ : kLessQ, cut);
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
    int how = !rejected ? kAll : !kDrafter ? kWithout : rejected == 1 ? kLessQ : kLessCutQ;
    Pair all = mass;
    if (!kDrafter || !rejected) {
        place();
        if (!kDrafter && rejected) {
            const int slice = (s1 - s0) * kVec;
            for (int i = tid; i < (slice + 31) / 32; i += kThreadsV) gone[i] = 0;
            __syncthreads();
            for (int i = cur + 1 + tid; i < n; i += kThreadsV) {
                const int x = a.tokens[c0 + i], v = x + off - s0 * kVec;
                if (a.parents[c0 + i] == cur && x >= 0 && x < V && v >= 0 && v < slice) atomicOr(&gone[v >> 5], 1u << (v & 31));
            }
            __syncthreads();
        }
        all = total(how, cut);
    }
    if (!positive(all)) {  // nothing is left of p: p itself
        how = kAll;
        all = total(kAll, zero);
    }
    float r = a.last[b];
    const bool bad_coin = !(r >= 0.0f && r < 1.0f);
    if (!(r >= 0.0f)) r = 0.0f;
    Pair goal = times(all, r);  // passed by a sum that is above it
    // The border: the CTA's slice that holds it, the warp's part in that, a thread's piece of that, the element. Where
    // rounding or r >= 1 puts the goal behind everything, the last one that weighs anything.
    const int owner = first_past(lane < ctas ? *cluster.map_shared_rank(&cta_sum[(pass - 1) & 1], lane) : zero, goal);
    if (rank == owner) {
        part_of(first_past(lane < kWarpsV ? warp_sum[lane] : zero, goal));
        const int piece = (k1 - k0 + kThreadsV - 1) / kThreadsV, a0 = min(k0 + tid * piece, k1), a1 = min(a0 + piece, k1);
        Pair s = zero;
        for (int k = a0; k < a1; ++k) {
            Pair x[kVec];
            careful(how, k, cut, x);
#pragma unroll
            for (int i = 0; i < kVec; ++i) add(s, x[i]);
        }
        const Pair upto = running_sum(s);
        __syncthreads();  // every warp has read warp_sum
        if (lane == 31) warp_sum[warp] = upto;
        if (tid == 0) {
            first_thread = kThreadsV;
            last_thread = -1;
        }
        __syncthreads();
        // what the warps in front hold
        const Pair in_front = running_sum(warp_sum[lane % kWarpsV]);
        const Pair front{__shfl_sync(kFull, in_front.hi, max(warp - 1, 0)), __shfl_sync(kFull, in_front.lo, max(warp - 1, 0))};
        if (warp) goal = less(goal, front);
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
                Pair x[kVec];
                careful(how, k, cut, x);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    add(t, x[i]);
                    if (!done && positive(x[i])) {
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

template <typename T, bool kDrafter>
cudaError_t launch_form(const VerifyArgs& a, cudaStream_t st) {
    auto* kernel = draft_verify_kernel<T, kDrafter>;
    constexpr int kVec = 16 / sizeof(T);
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = kDrafter ? cudaSuccess : allow_smem(allowed, kernel, kVerifyMaxVocab / 8 + 64);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Four CTAs fit on an SM: as many to a request as there is room for. (64 requests: 28.6 us; 512 threads, two to an SM
    // 29.6, 1024, one to an SM 48; a single small request 7.8, 8.4 and 9.5.)
    int ctas = kCtasMost;
    while (ctas > 1 && (int64_t)a.B * ctas > 4 * sms) ctas /= 2;
    const int64_t slice = (((a.V + 2 * kVec - 2) / kVec + ctas - 1) / ctas) * kVec;  // as if no row were aligned
    const size_t smem = kDrafter ? 0 : (size_t)(slice + 31) / 32 * 4;
    return launch_cluster(kernel, dim3((unsigned)(a.B * ctas)), dim3(kThreadsV), ctas, smem, st, a);
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, cudaStream_t st) {
    return a.draft ? launch_form<T, true>(a, st) : launch_form<T, false>(a, st);
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyArgs& a, cudaStream_t st) {
    if (a.ptype == IDX_FP32) return launch<float>(a, st);
    return a.ptype == IDX_BF16 ? launch<__nv_bfloat16>(a, st) : launch<__half>(a, st);
}

}  // namespace idx
