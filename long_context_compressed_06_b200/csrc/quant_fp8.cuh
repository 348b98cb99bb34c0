// quant_fp8.cuh -- one 8-element unit of the FP8 KV-row format (e4m3 codes with
// a UE8M0 exponent byte per 128 channels): its quantisation, shared by the row
// quantiser and the paged FP8 write, and its expansion in the attention kernels.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace csa {

// two floats -> two e4m3 codes (lo in the low byte), RNE, saturating
CSA_DEVINL uint32_t e4m3x2_rn_sat(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// a code of -0 (0x80) becomes +0
CSA_DEVINL uint32_t plus_zero(uint32_t w) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (((w >> (8 * i)) & 0xffu) == 0x80u) w &= ~(0xffu << (8 * i));
    return w;
}

// The 8 values f of this thread as codes (two words) under the exponent k of
// their 128-element block, the 16 threads of a block being 16 consecutive lanes
// that all take the call.
CSA_DEVINL uint2 quantize_fp8_unit(const float (&f)[8], int &k) {
    float amax = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) amax = fmaxf(amax, fabsf(f[q]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // smallest k with amax <= 448 * 2^k = 1.75 * 2^(8 + k), from amax's bit fields
    k = 0;
    if (amax > 0.f) {
        const uint32_t bits = __float_as_uint(amax);
        const int ef = (int)((bits >> 23) & 0xffu);
        if (ef == 0) {
            k = -124;  // subnormal absmax: far below the floor
        } else {
            const int E = ef - 127;
            k = (bits & 0x7fffffu) <= 0x600000u ? E - 8 : E - 7;  // mantissa <= 1.75 or above
        }
        k = k < -124 ? -124 : (k > 119 ? 119 : k);
    }
    const float inv = __uint_as_float((uint32_t)(127 - k) << 23);  // 2^-k, exact
    return make_uint2(plus_zero(e4m3x2_rn_sat(f[0] * inv, f[1] * inv) | (e4m3x2_rn_sat(f[2] * inv, f[3] * inv) << 16)),
                      plus_zero(e4m3x2_rn_sat(f[4] * inv, f[5] * inv) | (e4m3x2_rn_sat(f[6] * inv, f[7] * inv) << 16)));
}

// 8 e4m3 codes times 2^(e - 127) -> 8 bf16, exactly: e4m3 -> f16 is exact, the
// power-of-two scale is exact in fp32, and the product has at most 4
// significant bits inside bf16's range (the quantiser keeps e in [3, 246]).
CSA_DEVINL uint4 e4m3x8_bf16x8(uint2 raw, uint32_t e) {
    const float sc = __uint_as_float(e << 23);
    const uint32_t w[2] = {raw.x, raw.y};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
        const float lo = __half2float(__ushort_as_half((unsigned short)(h & 0xffffu))) * sc;
        const float hi = __half2float(__ushort_as_half((unsigned short)(h >> 16))) * sc;
        o[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace csa
