// pa_q8.cuh -- the 8-bit KV pool: code formats, the scale byte, conversions.
//
// A row (the 128 values of one token and kv head) is held as 128 one-byte
// codes and one scale byte s: value = code * 2^(s - 127).  s is 255 for a row
// that held a NaN or an infinity (every value reads back as NaN).  Finite rows
// have finite values: a code whose value would be 2^128, which bf16 does not
// hold, is the one below.
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

// Rows with a larger magnitude than this (bf16 bits) may hold numbers that round
// up to 2^128, as code 256 of scale 2^120 (E4M3) or 64 of 2^122 (INT8); the
// scales below end before 2^128, at 448 * 2^119 and 127 * 2^121.
template <int FMT>
constexpr uint32_t kQ8Top = FMT == PA_Q8_E4M3 ? 0x7f60u : 0x7f7eu;
// Such a row's pair of bf16, drawn in to the largest numbers that round to the
// codes below, 240 (from 247) and 63 (from 63.25).
template <int FMT>
__device__ __forceinline__ uint32_t q8_below_2_128(uint32_t w) {
    constexpr uint32_t most = FMT == PA_Q8_E4M3 ? 0x7f777f77u : 0x7f7d7f7du;
    asm("min.bf16x2 %0, %0, %1;\n\tmax.bf16x2 %0, %0, %2;" : "+r"(w) : "r"(most), "r"(most | 0x80008000u));
    return w;
}

// 2^(s - 127) in fp32; NaN for 255.
__device__ __forceinline__ float q8_scale(uint32_t s) {
    const uint32_t bits = s == 0 ? 0x00400000u : s << 23;
    return __uint_as_float(s == 255 ? 0x7fc00000u : bits);
}

// Four codes (one word) from two words of bf16 pairs and 2^-e.  The products are
// exact; the conversion (for INT8: adding 1.5 * 2^23, which leaves the integer
// in the low bits) is the one rounding.
template <int FMT>
__device__ __forceinline__ uint32_t q8_encode4(uint32_t lo, uint32_t hi, float inv) {
    uint32_t r;
    if (FMT == PA_Q8_E4M3) {
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(bf16lo(lo) * inv), "f"(bf16hi(lo) * inv), "f"(bf16lo(hi) * inv), "f"(bf16hi(hi) * inv));
    } else {
        constexpr float kMagic = 12582912.f;
        const uint32_t a = __float_as_uint(fmaf(bf16lo(lo), inv, kMagic)), b = __float_as_uint(fmaf(bf16hi(lo), inv, kMagic));
        const uint32_t c = __float_as_uint(fmaf(bf16lo(hi), inv, kMagic)), d = __float_as_uint(fmaf(bf16hi(hi), inv, kMagic));
        r = __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    }
    return r;
}

// Two pairs of INT8 codes of a word as f16x2, exactly, by the well-known way of
// making floats of small integers: the byte (offset by 128) is put under the
// exponent of 1024 and 1152 is subtracted, one permute and one packed subtract
// per pair.  A selector names its pair's bytes (0x4140: 0 and 1).
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

// Four codes of a word as two bf16 pairs, in order, times 2^e (a bf16 pair):
// exact wherever the value is a normal bf16 number.  INT8: bf16 holds 128 + the
// low seven bits, and 128 or 256 by the sign bit is subtracted.
template <int FMT>
__device__ __forceinline__ uint2 q8_to_bf16(uint32_t w, uint32_t scale) {
    uint32_t p[2];
    if (FMT == PA_Q8_E4M3) {
        uint32_t f[2];
        q8_to_f16<FMT>(w, f[0], f[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&f[j]));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[j]) : "f"(x.y), "f"(x.x));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t t = __byte_perm(w, 0x43434343u, j ? 0x4342 : 0x4140);
            asm("sub.bf16x2 %0, %1, %2;" : "=r"(p[j]) : "r"(t & 0xff7fff7fu), "r"(t & 0xff80ff80u));
        }
    }
    uint2 r;
    asm("mul.bf16x2 %0, %1, %2;" : "=r"(r.x) : "r"(p[0]), "r"(scale));
    asm("mul.bf16x2 %0, %1, %2;" : "=r"(r.y) : "r"(p[1]), "r"(scale));
    return r;
}

// 2^(s - 127) as a bf16 pair; NaN for 255.
__device__ __forceinline__ uint32_t q8_scale_bf16x2(uint32_t s) {
    const uint32_t h = s == 255 ? 0x7fc0u : s == 0 ? 0x0040u : s << 7;
    return h | (h << 16);
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
