// pa_q8.cuh -- the 8-bit KV pool: code formats, the scale byte, conversions.
//
// A row (the 128 values of one token and kv head) is held as 128 one-byte
// codes and one scale byte s: value = code * 2^(s - 127).  s is 255 for a row
// that held a NaN or an infinity (every value reads back as NaN).
//
// The scale is a power of two, so x * 2^-e is exact and a code is ONE rounding
// of the bf16 value (to nearest, ties to even); a code has at most 7
// significant bits, so reading it back as bf16 is exact as well.  A scale of
// amax / 127 would round twice (the scale, then the quotient), with ties that
// depend on how the quotient was computed.
#pragma once

#include <cuda_fp16.h>

#include "pa_internal.cuh"

namespace pa {

constexpr int Q8_D = 128;  // values of a row

// The smallest exponent e for which amax * 2^-e stays within the codes' range
// (448 = 1.75 * 2^8, or 127 = 127/64 * 2^6), from amax's bf16 bits; at least
// -126, so that 2^e and 2^-e are both normal fp32 numbers.
template <int FMT>
__device__ __forceinline__ int q8_exponent(uint32_t amax_bits) {
    const int p = (int)(amax_bits >> 7) - 127, m = (int)(amax_bits & 0x7f);
    const int e = FMT == PA_Q8_E4M3 ? p - 8 + (m > 0x60 ? 1 : 0) : p - 6 + (m > 0x7e ? 1 : 0);
    return max(e, -126);
}

// 2^(s - 127) in fp32; NaN for 255.
__device__ __forceinline__ float q8_scale(uint32_t s) {
    const uint32_t bits = s == 0 ? 0x00400000u : s << 23;
    return __uint_as_float(s == 255 ? 0x7fc00000u : bits);
}

// Four codes (one word) from four scaled values.
template <int FMT>
__device__ __forceinline__ uint32_t q8_encode4(float a, float b, float c, float d) {
    uint32_t r;
    if (FMT == PA_Q8_E4M3) {
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
    } else {
        const uint32_t ab = __byte_perm((uint32_t)__float2int_rn(a), (uint32_t)__float2int_rn(b), 0x0040);
        const uint32_t cd = __byte_perm((uint32_t)__float2int_rn(c), (uint32_t)__float2int_rn(d), 0x0040);
        r = __byte_perm(ab, cd, 0x5410);
    }
    return r;
}

// Two pairs of INT8 codes of a word as f16x2, exactly: the byte (offset by 128)
// is put under the exponent of 1024 and 1152 is subtracted, one permute and one
// packed subtract per pair.  A selector names its pair's bytes (0x4140: 0 and 1).
template <uint32_t LO, uint32_t HI>
__device__ __forceinline__ void q8_int8_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, LO), b = __byte_perm(u, 0x64646464u, HI);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// The codes in bytes 0, 1 (lo) and 2, 3 (hi) of a word as f16x2, exactly.
template <int FMT>
__device__ __forceinline__ void q8_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (FMT == PA_Q8_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\t"
            "mov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        q8_int8_to_f16<0x4140, 0x4342>(w, lo, hi);
    }
}

// Host checks shared by the entry points over an 8-bit pool.
inline pa_status q8_check_pool(int32_t format, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                               int32_t num_blocks) {
    if (format != PA_Q8_E4M3 && format != PA_Q8_INT8) return fail(PA_ERR_INVALID_ARG, "unknown 8-bit format %d", format);
    if (num_kv_heads <= 0) return fail(PA_ERR_INVALID_ARG, "num_kv_heads must be positive");
    if (head_dim != Q8_D) return fail(PA_ERR_UNSUPPORTED, "head_dim %d (only 128)", head_dim);
    if (block_size <= 0 || block_size % 16)
        return fail(PA_ERR_UNSUPPORTED, "block_size %d (must be a positive multiple of 16)", block_size);
    if (num_blocks <= 0) return fail(PA_ERR_INVALID_ARG, "num_blocks must be positive");
    // Rows (token, head) are TMA coordinates and slots are int32.
    if ((int64_t)num_blocks * block_size > 0x7fffffffLL / num_kv_heads)
        return fail(PA_ERR_UNSUPPORTED, "pool of %d blocks too large for 32-bit row indices", num_blocks);
    return PA_OK;
}

}  // namespace pa
