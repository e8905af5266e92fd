// kv.cuh -- the 8-bit paged KV cache's layout (idx_kv_layout) and element conversions, shared by
// the store and the attention kernels.
#pragma once

#include "common.cuh"

namespace idx {

constexpr int kKvBlock = 16;                 // tokens that share a scale
constexpr int kKvEMin = -32, kKvEMax = 48;   // range of a scale's exponent

__host__ __device__ constexpr int64_t kv_head_bytes(int P, int D) { return 2ll * P * D + 16; }

// 2^e as fp32, e in [-126, 127]
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// two e4m3 codes (low byte first) -> two fp16 (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t d;
    asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}" : "=r"(d) : "r"(two));
    return d;
}
// four codes -> two pairs
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %2;\n cvt.rn.f16x2.e4m3x2 %0, t;\n cvt.rn.f16x2.e4m3x2 %1, u;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
// NaN codes (0x7f, 0xff) among four replaced by 0; whether there was one
__device__ __forceinline__ bool clear_nan_codes(uint32_t& four) {
    const uint32_t hit = ((four & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // 0x7f + 1 carries into bit 7
    four &= ~((hit >> 7) * 255u);
    return hit != 0;
}
// two fp32 -> two e4m3 codes (a in the low byte), nearest even, saturating
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float a, float b) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(d) : "f"(a), "f"(b));
    return d;
}

}  // namespace idx
