// kv_store.cu -- K and V rows into the 8-bit paged KV cache (idx_kv_store).
//
// A scale belongs to 16 tokens of a page, one head and one side (K or V): 2^E with the least E
// for which the largest magnitude m * 2^e (1 <= m < 2) is at most 448 * 2^E = 1.75 * 2^(E+8), that is
// E = e - 8, or e - 7 for m > 1.75. Powers of two cost e4m3 no precision (its relative step is
// the same in every binade) and make scaling exact, so that appending to a block, whose kept codes
// take the larger scale by a shift of their exponents, gives what storing the block at once
// would (but for values that become subnormal), and the bytes are the same on any machine.
//
// One warp owns what a call writes into one block of one head: a run of at most 16 adjacent rows.
// It holds them in registers (16-byte loads, 16 or 8 lanes a row), so that the rows are read
// once: maximum, scale, codes.
// Measured in replayed graphs (bf16, 8 heads, D = 128): 8192 rows of a prompt 11.2 us, 4.5 TB/s of rows read and codes
// written (floor 7.4 us at the measured copy rate); 64 single rows 3.4 us, launch and one chain of loads (a call from the
// host takes 10 us more).
#include "kernels.h"
#include "kv.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace idx {

namespace {

template <bool kHalf>
__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kHalf) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = bf16_lo(u[i]);
            x[2 * i + 1] = bf16_hi(u[i]);
        }
    }
}

// Least E in [kKvEMin, kKvEMax] with amax <= 448 * 2^E; amax finite, >= 0.
__device__ __forceinline__ int block_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127;  // subnormals end below kKvEMin all the same
    const int E = (u & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7;
    return min(max(E, kKvEMin), kKvEMax);
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(128) kv_store_kernel(const KvStoreArgs a, int window) {
    constexpr int kLanes = D / 8;           // lanes of a row, 8 values each
    constexpr int kRows = 32 / kLanes;      // rows of one load
    constexpr int kSteps = kKvBlock / kRows;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int head = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int64_t w0 = (int64_t)blockIdx.x * window;  // this CTA takes the runs that begin in rows w0 .. w0 + window - 1
    const int64_t slots_total = a.num_pages * a.page_size;
    // lane i holds row w0 - 1 + i: the row before the window, the window, and what a run may reach behind it
    const int64_t rr = w0 + lane - 1;
    const int64_t slot = (rr >= 0 && rr < a.n_rows && lane <= window + kKvBlock - 1) ? a.slot_mapping[rr] : -1;
    const int64_t prev = __shfl_up_sync(kFull, slot, 1);
    const bool live = slot >= 0 && slot < slots_total, mine = lane >= 1 && lane <= window;
    const bool mates = lane >= 1 && live && prev >= 0 && prev / kKvBlock == slot / kKvBlock;
    const unsigned on = __ballot_sync(kFull, mates && slot > prev);  // rows that continue their predecessor's run
    if (head == 0 && mine && ((slot >= slots_total) || (mates && slot <= prev)))
        report(a.dev_status, IDX_STATUS_BAD_SLOT);
    unsigned begin = __ballot_sync(kFull, mine && live && !mates);
    if (head >= a.kv_heads) return;
    for (; begin; begin &= begin - 1) {
        const int first = __ffs(begin) - 1;  // lane of the run's first row
        const unsigned stop = ~(on >> (first + 1));
        const int n = __ffs(stop);           // rows of the run, 16 at most
        const int64_t r0 = w0 + first - 1, s0 = __shfl_sync(kFull, slot, first);
        const int f = (int)(s0 % kKvBlock);
        const int off = (int)(slot - s0) + f;  // in-block offset of this lane's row, where it is one of the run
        const int P = a.page_size;
        const int64_t page = s0 / P;
        uint8_t* base = a.pool + page * a.page_stride + head * kv_head_bytes(P, D);
        const int blk = (int)(s0 % P) / kKvBlock;
        uint8_t* scale = base + 2ll * P * D + 2 * blk;
        uint8_t* tok = base + (int64_t)blk * kKvBlock * 2 * D;
        const int c = lane % kLanes, sub = lane / kLanes;

        const int old_k = f ? (int)scale[0] - 127 : kKvEMin, old_v = f ? (int)scale[1] - 127 : kKvEMin;
        uint4 raw[2][kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = i * kRows + sub;
            raw[0][i] = raw[1][i] = make_uint4(0, 0, 0, 0);
            if (r < n) {
                raw[0][i] = *(reinterpret_cast<const uint4*>(a.k + (r0 + r) * a.k_row_stride + head * a.k_head_stride) + c);
                raw[1][i] = *(reinterpret_cast<const uint4*>(a.v + (r0 + r) * a.v_row_stride + head * a.v_head_stride) + c);
            }
        }
        bool nan = false;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                float x[8];
                unpack8<kHalf>(raw[side][i], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float m = fabsf(x[j]);
                    amax = fmaxf(amax, m < __int_as_float(0x7f800000) ? m : 0.0f);
                    nan |= x[j] != x[j];
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            const int old = min(max(side ? old_v : old_k, kKvEMin), kKvEMax);
            const int E = max(block_exponent(amax), old);
            if (f && E > old) {  // the kept tokens take the larger scale
                const float g = pow2f(old - E);
                for (int t = sub; t < f; t += kRows) {
                    uint2* p = reinterpret_cast<uint2*>(tok + (int64_t)t * 2 * D + side * D) + c;
                    uint2 w = *p;
                    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t lo, hi;
                        e4m3x4_to_f16x4(u[j], lo, hi);
                        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                        u[j] = f32x2_to_e4m3x2(x.x * g, x.y * g) | f32x2_to_e4m3x2(y.x * g, y.y * g) << 16;
                    }
                    *p = w;
                }
            }
            const float inv = pow2f(-E);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int r = i * kRows + sub;
                const int at = __shfl_sync(kFull, off, (first + r) & 31);
                float x[8];
                unpack8<kHalf>(raw[side][i], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] == x[j] ? x[j] * inv : 0.0f;
                uint2 w;
                w.x = f32x2_to_e4m3x2(x[0], x[1]) | f32x2_to_e4m3x2(x[2], x[3]) << 16;
                w.y = f32x2_to_e4m3x2(x[4], x[5]) | f32x2_to_e4m3x2(x[6], x[7]) << 16;
                if (r < n) reinterpret_cast<uint2*>(tok + (int64_t)at * 2 * D + side * D)[c] = w;
            }
            if (lane == 0) scale[side] = (uint8_t)(E + 127);
        }
        if (__any_sync(kFull, nan) && lane == 0) report(a.dev_status, IDX_STATUS_BAD_VALUE);
    }
}

}  // namespace

cudaError_t launch_kv_store(const KvStoreArgs& a, cudaStream_t st) {
    // Few rows (decode): a CTA per row, for the runs are one row each. Many rows (prompts): most rows continue a
    // run, so a CTA looks at 16 (8192 rows, 8 heads: 11.1 us against 28.0 with a CTA per row).
    const int window = a.n_rows >= 1024 ? 16 : 1;
    const dim3 grid((unsigned)((a.n_rows + window - 1) / window), (unsigned)((a.kv_heads + 3) / 4)), block(128);
    if (a.head_dim == 128)
        return a.ftype == IDX_FP16 ? launch_pdl(kv_store_kernel<128, true>, grid, block, 0, st, a, window)
                                   : launch_pdl(kv_store_kernel<128, false>, grid, block, 0, st, a, window);
    return a.ftype == IDX_FP16 ? launch_pdl(kv_store_kernel<64, true>, grid, block, 0, st, a, window)
                               : launch_pdl(kv_store_kernel<64, false>, grid, block, 0, st, a, window);
}

}  // namespace idx
