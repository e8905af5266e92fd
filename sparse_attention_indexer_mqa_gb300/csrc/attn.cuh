// attn.cuh -- what the attention kernels over the 8-bit paged KV cache share: the row rules, the
// numbers of the running softmax and the output writes.
//
// The softmax that every kernel keeps. With s = q . k_code (fp32 sum), c = softmax_scale * log2(e)
// * (q's power of two) * 2^Ek and Ev the exponent of the key's V block,
//     u = s * c + Ev,   p' = 2^(u - m + kShift),   O += p' * v_code,   l += p' * 2^-Ev:
// V's scale is part of the weight, so both products run on bare codes and nothing has to be
// scaled element by element. m follows the largest u; it is raised only when a u passes it by more than
// kLazy, since raising it means rescaling O and l (with 3 some row of a warp's 32 was raised in every
// second step of 128 keys, by the counter of O's loads in a 4096-token prompt; with 8 in few). p' <=
// 2^(kShift + kLazy) = 2^15 stays in fp16's range. What is rounded to fp16 is the weight times 2^Ev: down to 2^-21 of
// the row's largest such product it keeps fp16's full 11 bits, below that an absolute 2^-32 of it (so a key of large
// weight in a block of small V can lose its V beside a block of large V).
//     out = O / l,   lse = ln 2 * (m - kShift + log2 l).
// -32 <= Ev <= 48, so that in fp32, in which l is summed, p' and p' * 2^-Ev can only underflow where the weight is
// below 2^-46 of the row's largest.
//
// A NaN code. Of K it makes the scores of its key NaN, which a row that does not see the key drops with the
// score. Of V it would come through the product at weight 0 too, so where a unit's rows see unlike numbers of
// keys (the diagonal of a causal unit) V's NaN codes are taken out of the steps that some row does not see whole, the
// lowest such key is kept, and rows that see it are NaN at the end. Rows of a tree see sets that do not contain one
// another, so a bit for each of its nodes is kept instead. Everywhere else all rows see what was loaded and the product
// does it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.h"
#include "kv.cuh"

namespace idx {

constexpr float kShift = 7.0f, kLazy = 8.0f;
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two fp32 operations in one instruction, each rounded as by itself
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
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? neg_inf() : kLn2 * (m - kShift + log2f(l));
}

// A block's two scale bytes (K low, V high; 127 + E): 2^Ek, and Ev. Bytes that the store does not write
// are taken as the nearest that it does.
__device__ __forceinline__ uint32_t scale_byte(uint32_t e) {
    return min(max(e & 255u, (uint32_t)(127 + kKvEMin)), (uint32_t)(127 + kKvEMax));
}
__device__ __forceinline__ float k_scale(uint32_t two) { return __uint_as_float(scale_byte(two) << 23); }
__device__ __forceinline__ float v_exponent(uint32_t two) { return (float)((int)scale_byte(two >> 8) - 127); }

// A sequence's rows: its first query row and how many, or nq = -1 if it breaks its bounds.
struct SeqRows {
    int64_t t0;
    int32_t nq, len;
};
__device__ __forceinline__ SeqRows seq_rows(const AttnArgs& a, int b) {
    SeqRows s;
    const int32_t c0 = a.cu_seqlens_q[b], c1 = a.cu_seqlens_q[b + 1];
    s.len = a.seq_lens_k[b];
    s.t0 = c0;
    s.nq = c1 - c0;
    if (c0 < 0 || c1 < c0 || c1 > a.T || s.nq > a.max_q_len || s.len < 0 || s.len > a.max_seq_len_k) s.nq = -1;
    return s;
}

// The sequence that owns query row t, or -1, found by a whole warp: each round cuts the range by 32 with one round
// trip to memory, where a binary search takes five.
__device__ __forceinline__ int warp_seq_of_query(const AttnArgs& a, int64_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.B;  // cu[lo] <= t < cu[hi], if t is in any sequence
    bool in = true;
    for (bool first = true; first || hi - lo > 1; first = false) {
        const int step = (hi - lo + 31) / 32;
        const int at = min(lo + (lane + 1) * step, hi);
        const int32_t c = a.cu_seqlens_q[at];
        if (first) in = t >= a.cu_seqlens_q[0] && t < a.cu_seqlens_q[a.B];
        const unsigned above = __ballot_sync(kFull, c > t);  // ends of parts that lie behind t; the last one does
        const int part = above ? __ffs(above) - 1 : 31;
        hi = min(lo + (part + 1) * step, hi);
        lo = min(lo + part * step, hi - 1);
        if (!in) break;
    }
    return in ? lo : -1;
}

// A tree of drafted tokens (idx_attn_tree). The last nq keys of a sequence are its nodes, the keys in front of
// them are seen by every row. Bits of the 64 keys from position `front` + j0 on, set where a row with this mask sees
// the key: j0 < 0 for keys in front of the tree, nothing behind its end.
__device__ __forceinline__ uint64_t tree_window(const uint64_t* mask, int words, int nq, int j0) {
    if (j0 <= -64) return ~0ull;
    uint64_t w = 0;
    if (j0 < 0) {
        w = mask[0] << -j0 | ((1ull << -j0) - 1);
    } else {
        const int at = j0 >> 6, by = j0 & 63;
        if (at < words) w = mask[at] >> by;
        if (by && at + 1 < words) w |= mask[at + 1] << (64 - by);
    }
    const int left = nq - j0;
    return left >= 64 ? w : left <= 0 ? 0 : w & ((1ull << left) - 1);
}
// Whether a row with this mask sees a node whose bit is set in `nodes`.
__device__ __forceinline__ bool tree_sees(const uint64_t* mask, int words, int nq, const uint32_t* nodes) {
    bool hit = false;
    for (int w = 0; w < (nq + 63) / 64; ++w)
        hit |= (tree_window(mask, words, nq, 64 * w) & (nodes[2 * w] | (uint64_t)nodes[2 * w + 1] << 32)) != 0;
    return hit;
}

// Power of two that brings a row of q with the given largest magnitude into fp16's range (its
// largest value to [2^14, 2^15)), and the exponent it takes away. fp16 rows stay as they are.
template <bool kHalf>
__device__ __forceinline__ int q_exponent(float amax) {
    if constexpr (kHalf) return 0;
    const int e = (int)(__float_as_uint(amax) >> 23) - 127;
    return amax > 0.0f ? max(e, -100) - 14 : 0;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kHalf>
__device__ __forceinline__ float2 load_pair(uint32_t w) {
    if constexpr (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool kHalf>
__device__ __forceinline__ uint32_t store_pair(float x, float y) {
    if constexpr (kHalf) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace idx
