// attn_tc.cuh -- the parts of the tensor-memory attention kernel (attn_tc.cu): operand tiles, MMA issue, the
// rows' way in and out. A tile is 128 query rows by 128 keys. Operands are fp16, K-major with the
// 128-byte swizzle: Q [D/64][128 rows][128 B], K [D/64][128 keys][128 B], V transposed
// [2][D dims][128 B] (64 keys to a row).
#pragma once

#include "attn.cuh"
#include "tc.cuh"

namespace idx {

constexpr int kRowsT = 128;   // rows of a tile
constexpr int kKeysT = 128;   // keys of a step

template <int D>
constexpr int kOutRow = 4 * D + 16;  // bytes of a staged row of results

// Pauses between tests of a barrier (ns). None was measurably better or worse from 0 to 200.
constexpr int kNsIssue = 0, kNsSoft = 0, kNsConv = 20;

// Bounded wait of a whole warp: every lane gets the same answer.
template <int kNs>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(kFull, tc::mbar_spin<kNs>(bar, parity));
}

// Where 8 consecutive dims (chunk i) of q and k lie in the operand tiles: any order serves, and this one
// lets 8 lanes that convert one key's consecutive 16-byte pieces write 8 different chunks.
template <int D>
__device__ __forceinline__ constexpr int dims_sub(int i) { return D == 128 ? i & 1 : 0; }
template <int D>
__device__ __forceinline__ constexpr int dims_chunk(int i) { return D == 128 ? i >> 1 : (i >> 1) + 4 * (i & 1); }

// A converter thread ct's share (of 128): 8 lanes take consecutive pieces of a row, so that a memory
// request touches few lines. K: 16-byte piece kp of keys k_key + i * kKeyStep. V: kVB bytes from dim
// kVB * dg of keys 8 * kg .. + 7; dim kVB * dg + y goes to row 8 * y + dg of the transposed tile (8
// lanes, 8 chunks).
template <int D>
struct ConvShare {
    static constexpr int kPieces = D / 16, kVB = D / 8, kKeyStep = D == 128 ? 16 : 32;
    int kp, k_key, kg, dg;
    __device__ __forceinline__ explicit ConvShare(int ct) {
        const int lane = ct & 31, cw = ct >> 5;
        kp = D == 128 ? lane & 7 : lane & 3;
        k_key = D == 128 ? (lane >> 3) + 4 * cw : (lane >> 3) + (lane & 4) + 8 * cw;
        kg = (lane >> 3) + 4 * cw;
        dg = lane & 7;
    }
};

// One 16-byte piece of K (piece kp of `key`) as fp16 into the K tile; f != 0: times the pair f.
template <int D>
__device__ __forceinline__ void write_k_piece(uint8_t* tile, const uint4& raw, int key, int kp, uint32_t f) {
    uint4 lo, hi;
    e4m3x4_to_f16x4(raw.x, lo.x, lo.y);
    e4m3x4_to_f16x4(raw.y, lo.z, lo.w);
    e4m3x4_to_f16x4(raw.z, hi.x, hi.y);
    e4m3x4_to_f16x4(raw.w, hi.z, hi.w);
    if (f) {
        lo.x = mul_f16x2(lo.x, f); lo.y = mul_f16x2(lo.y, f);
        lo.z = mul_f16x2(lo.z, f); lo.w = mul_f16x2(lo.w, f);
        hi.x = mul_f16x2(hi.x, f); hi.y = mul_f16x2(hi.y, f);
        hi.z = mul_f16x2(hi.z, f); hi.w = mul_f16x2(hi.w, f);
    }
    uint8_t* row = tile + key * 128;
    *reinterpret_cast<uint4*>(row + dims_sub<D>(0) * (kKeysT * 128) + ((dims_chunk<D>(2 * kp) ^ (key & 7)) << 4)) = lo;
    *reinterpret_cast<uint4*>(row + dims_sub<D>(1) * (kKeysT * 128) + ((dims_chunk<D>(2 * kp + 1) ^ (key & 7)) << 4)) = hi;
}

// A block of V (kVB dims of 8 keys) as fp16, transposed, into the V tile; fold: keys 2i, 2i + 1 times the
// pair f[i].
template <int D>
__device__ __forceinline__ void write_v_block(uint8_t* tile, const uint4 (&rv)[8], int kg, int dg, bool fold,
                                              const uint32_t (&f)[4]) {
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = w == 0 ? rv[i].x : w == 1 ? rv[i].y : w == 2 ? rv[i].z : rv[i].w;
        uint32_t t[4][4];  // [dim][pair of keys]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            e4m3x4_to_f16x4(__byte_perm(u[2 * i], u[2 * i + 1], 0x5140), t[0][i], t[1][i]);
            e4m3x4_to_f16x4(__byte_perm(u[2 * i], u[2 * i + 1], 0x7362), t[2][i], t[3][i]);
        }
        if (fold) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int i = 0; i < 4; ++i) t[y][i] = mul_f16x2(t[y][i], f[i]);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int row = 8 * (4 * w + y) + dg;  // of dim kVB * dg + 4 * w + y
            *reinterpret_cast<uint4*>(tile + (kg >> 3) * (D * 128) + row * 128 + (((kg & 7) ^ dg) << 4)) =
                make_uint4(t[y][0], t[y][1], t[y][2], t[y][3]);
        }
    }
}

// A warp's 32 rows of q as fp16 into rows first .. first + 31 of the Q tile (zeros where a row does not exist or is not
// finite); src: each lane's row. Returns the lane's row's factor: softmax_scale * log2(e) * (the power of two taken
// out), -1 for a row that is not finite. D/8 lanes take a row, so that a request touches whole lines; with a row to a thread
// a unit's start took 8 us where every SM was loading.
template <int D, bool kHalf>
__device__ __forceinline__ float write_q_rows(uint8_t* tile, const uint16_t* src, bool real, int first, float scale) {
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kBatch = 4;
    const int lane = threadIdx.x & 31, i = lane % kLanes, sub = lane / kLanes;
    const unsigned exist = __ballot_sync(kFull, real);
    const uint32_t lo = (uint32_t)reinterpret_cast<uintptr_t>(src), hi = (uint32_t)(reinterpret_cast<uintptr_t>(src) >> 32);
    float mine = 0.0f;
    if (!exist) {  // the other form of the loop below, for warps that have something else to do
#pragma unroll 1
        for (int r = sub; r < 32; r += kAtOnce)
            *reinterpret_cast<uint4*>(tile + dims_sub<D>(i) * (kRowsT * 128) + (first + r) * 128 +
                                      ((dims_chunk<D>(i) ^ ((first + r) & 7)) << 4)) = make_uint4(0, 0, 0, 0);
        return mine;
    }
#pragma unroll 1
    for (int s0 = 0; s0 < kLanes; s0 += kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int s = 0; s < kBatch; ++s) {
            const int r = (s0 + s) * kAtOnce + sub;
            const uint32_t l = __shfl_sync(kFull, lo, r), h = __shfl_sync(kFull, hi, r);
            const uint4* row = reinterpret_cast<const uint4*>((uintptr_t)h << 32 | l);
            w[s] = make_uint4(0, 0, 0, 0);
            if (exist >> r & 1u) w[s] = row[i];
        }
#pragma unroll
        for (int s = 0; s < kBatch; ++s) {
            const int r = (s0 + s) * kAtOnce + sub, row = first + r;
            uint32_t u[4] = {w[s].x, w[s].y, w[s].z, w[s].w};
            float amax = 0.0f;
            bool odd = false;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float2 f = load_pair<kHalf>(u[x]);
                odd |= !(fabsf(f.x) < __int_as_float(0x7f800000)) || !(fabsf(f.y) < __int_as_float(0x7f800000));
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            const unsigned odds = __ballot_sync(kFull, odd);
            odd = (odds >> (sub * kLanes) & (kLanes == 32 ? ~0u : (1u << kLanes) - 1)) != 0;
            if constexpr (!kHalf) {
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            }
            const int e = odd ? 0 : q_exponent<kHalf>(amax);
            const float up = pow2f(-e);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (odd) u[x] = 0;
                if constexpr (!kHalf) {
                    const float2 f = load_pair<kHalf>(u[x]);
                    u[x] = half2_bits(f.x * up, f.y * up);
                }
            }
            *reinterpret_cast<uint4*>(tile + dims_sub<D>(i) * (kRowsT * 128) + row * 128 + ((dims_chunk<D>(i) ^ (row & 7)) << 4)) =
                make_uint4(u[0], u[1], u[2], u[3]);
            const float f = __shfl_sync(kFull, odd ? -1.0f : scale * kLog2e * pow2f(e), lane % kAtOnce * kLanes);
            if (lane / kAtOnce == s0 + s) mine = f;
        }
    }
    return mine;
}

// S = Q K^T and O (+)= P V of a step, by one lane of the (converged) warp that calls. P lies in the
// first half of S's columns, as fp16.
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t tm_s, uint32_t q_tile, uint32_t k_tile, uint64_t* done) {
    tc::tc_fence_after();
    const uint64_t qd = tc::smem_desc_sw128(q_tile), kd = tc::smem_desc_sw128(k_tile);
    if (tc::elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = ((k / 4) * (128 * 128) + (k % 4) * 32) >> 4;  // in the descriptor's 16-byte units
            tc::mma_f16(tm_s, qd + at, kd + at, tc::idesc_f16(kRowsT, kKeysT), k > 0);
        }
        tc::mma_commit(done);
    }
    __syncwarp();
}
template <int D>
__device__ __forceinline__ void issue_outputs(uint32_t tm_o, uint32_t tm_p, uint32_t v_tile, bool accumulate,
                                              uint64_t* done) {
    tc::tc_fence_after();
    const uint64_t vd = tc::smem_desc_sw128(v_tile);
    if (tc::elect_one()) {
#pragma unroll
        for (int k = 0; k < kKeysT / 16; ++k)
            tc::mma_f16_ta(tm_o, tm_p + 8 * k, vd + (((k / 4) * (D * 128) + (k % 4) * 32) >> 4),
                           tc::idesc_f16(kRowsT, D), accumulate || k > 0);
        tc::mma_commit(done);
    }
    __syncwarp();
}

// A warp's rows out of tensor memory (tm_o: the warp's lanes): the result, or the split's part of it. some: O was
// written at all. nan: a NaN code of V among the row's keys. Column 8y + x of O is dim (D/8) * x + y, so 32 columns are 4 dims of each x.
// The rows pass through shared memory (32 * kOutRow<D> bytes of the warp's own, from K's tile on: the last product has
// read it, and without keys nothing writes there), so that a request writes whole rows: 8 bytes of each of 32 rows a request took 4 us where every SM was writing.
template <int D, bool kHalf>
__device__ __forceinline__ void store_rows(const AttnArgs& a, uint32_t tm_o, uint8_t* stage, bool some, bool real, int64_t tok, int hq,
                                           int z, float m, float l, bool nan) {
    const bool part = a.n_split > 1;
    const float g = nan ? __int_as_float(0x7fc00000) : part ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
    const int64_t pr = ((int64_t)z * a.T + tok) * a.q_heads + hq;
    const int lane = threadIdx.x & 31;
    uint8_t* own = stage + lane * kOutRow<D>;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        __syncwarp();
        if (some) {
            tc::tmem_ld32(tm_o + 32 * c, r);
            tc::tmem_ld_wait();
        }
        if (!(some && l != 0.0f)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            float v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] = __uint_as_float(r[8 * y + x]) * g;
            const int dim = D / 8 * x + 4 * c;
            if (part)
                *reinterpret_cast<float4*>(own + 4 * dim) = make_float4(v[0], v[1], v[2], v[3]);
            else
                *reinterpret_cast<uint2*>(own + 2 * dim) = make_uint2(store_pair<kHalf>(v[0], v[1]), store_pair<kHalf>(v[2], v[3]));
        }
    }
    // where each lane's row goes; a part without keys is not written
    uint8_t* to = part ? reinterpret_cast<uint8_t*>(a.part_o + pr * D)
                       : reinterpret_cast<uint8_t*>(a.out + tok * a.out_row_stride + (int64_t)hq * a.out_head_stride);
    const unsigned go = __ballot_sync(kFull, real && (!part || l != 0.0f));
    __syncwarp();  // every lane has staged its row
    const uint32_t lo = (uint32_t)reinterpret_cast<uintptr_t>(to), hi = (uint32_t)(reinterpret_cast<uintptr_t>(to) >> 32);
    const int pieces = part ? D / 4 : D / 8, at_once = 32 / pieces, i = lane % pieces;
#pragma unroll 4
    for (int r0 = 0; r0 < 32; r0 += at_once) {
        const int r = r0 + lane / pieces;
        const uint32_t ll = __shfl_sync(kFull, lo, r), hh = __shfl_sync(kFull, hi, r);
        if (go >> r & 1u)
            reinterpret_cast<uint4*>((uintptr_t)hh << 32 | ll)[i] = *reinterpret_cast<const uint4*>(stage + r * kOutRow<D> + 16 * i);
    }
    if (real) {
        if (part)
            a.part_ml[pr] = make_float2(m, l);
        else if (a.lse)
            a.lse[tok * a.q_heads + hq] = lse_of(m, l);
    }
}

}  // namespace idx
