// pa_rope.cu -- per-head norm and rotation of q and k, and the store of the
// rotated keys and of the values into the pool.
//
// What it computes, per head x of 128 values at position p: optionally
//   x <- x * rsqrt(mean(x^2) + eps) * weight,
// then the first R values in pairs (x1, x2) = (x[i], x[i + R/2]) or, interleaved,
// (x[2i], x[2i+1]), i < R/2:
//   (x1 cos a - x2 sin a, x2 cos a + x1 sin a) * gain,  a = 2 pi p f_i,
// f_i in turns per position; everything in fp32, rounded once to bf16.
//
// The angle: f_i is a fraction of 2^64 and p * f_i is taken modulo 2^64, so the
// turns are exact for every 32-bit position; the signed result is rounded once
// to fp32 (an angle error of at most 2^-25 pi) before sincospif.  The product in
// fp32 would be off by 4e-3 at position 10^5 and by 3e-2 at 10^6.
//
// Layout: eight lanes per head, two 16-byte chunks a lane, chosen so that both
// halves of a pair are in one lane: chunks 8l and R/2 + 8l of the rotated part
// (split halves), 16l and 16l + 8 otherwise.  A warp's four lane groups take four
// heads and share the token's 64 angles: each lane evaluates two and gets its
// eight by shuffles.
#include <math.h>

#include <algorithm>

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int ROPE_D = 128;
constexpr int ROPE_THREADS = 256;
constexpr unsigned FULL = 0xffffffffu;

struct RopeArgs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    __nv_bfloat16 *out_q, *out_k;          // out_k: rotated keys by token (no store)
    int64_t out_q_stride, out_k_stride;
    __nv_bfloat16 *k_cache, *v_cache;      // null: no store
    const int32_t *slots;
    int64_t num_slots;
    const int32_t *positions;
    const unsigned long long *freqs;
    const __nv_bfloat16 *wq, *wk;          // null: no norm
    float gain, eps;
    int32_t tokens, Hq, Hkv, heads;        // heads: all that a token moves
    int32_t rotary, parts;                 // parts: units per token
    DevError *err;
};

__device__ __forceinline__ uint4 ld_row16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
    x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
    x[4] = bf16lo(w.z); x[5] = bf16hi(w.z); x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
}

__device__ __forceinline__ uint32_t pack2bf(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2bf(x[0], x[1]), pack2bf(x[2], x[3]), pack2bf(x[4], x[5]), pack2bf(x[6], x[7]));
}

// A unit is one token and U groups of four heads: its q heads, then its k heads,
// then (store) its v heads.
template <bool INTER, int U>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const __grid_constant__ RopeArgs a) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, l = lane & 7, grp = lane >> 3;
    const bool rot = 16 * l < a.rotary;
    const int c0 = (INTER || !rot) ? 16 * l : 8 * l;
    const int c1 = (INTER || !rot) ? 16 * l + 8 : a.rotary / 2 + 8 * l;
    const uint32_t nunits = (uint32_t)a.tokens * (uint32_t)a.parts;
    const uint32_t wstride = gridDim.x * (ROPE_THREADS / 32);
    // The two pairs whose angle this lane evaluates.
    unsigned long long f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) f[e] = rot ? __ldg(a.freqs + 8 * l + 2 * grp + e) : 0ull;
    for (uint32_t unit = blockIdx.x * (ROPE_THREADS / 32) + (threadIdx.x >> 5); unit < nunits; unit += wstride) {
        const uint32_t token = unit / (uint32_t)a.parts;
        const int h0 = (int)(unit - token * (uint32_t)a.parts) * (4 * U) + grp;
        const long long pos = __ldg(a.positions + token);
        int64_t slot = 0;
        if (a.k_cache != nullptr) {
            slot = __ldg(a.slots + token);
            if (slot >= a.num_slots) {
                if (h0 == 0 && l == 0) record_error(a.err, PA_DEV_BAD_SLOT, token);
                slot = -1;
            }
        }
        uint4 w0[U], w1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + 4 * u;
            if (h >= a.heads || (h >= a.Hq && slot < 0)) continue;
            const __nv_bfloat16 *src = h < a.Hq            ? a.q + token * a.q_stride + (int64_t)h * ROPE_D
                                       : h < a.Hq + a.Hkv ? a.k + token * a.k_stride + (int64_t)(h - a.Hq) * ROPE_D
                                                          : a.v + token * a.v_stride + (int64_t)(h - a.Hq - a.Hkv) * ROPE_D;
            w0[u] = ld_row16(src + c0);
            w1[u] = ld_row16(src + c1);
        }
        float cs[8], sn[8];
        {
            float c2[2], s2[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const long long turns = (long long)((unsigned long long)pos * f[e]);  // in 2^-64, -1/2 .. 1/2
                sincospif((float)turns * 0x1p-63f, &s2[e], &c2[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int from = (e >> 1) * 8 + l;
                const float g = rot ? a.gain : 1.f;
                cs[e] = __shfl_sync(FULL, c2[e & 1], from) * g;
                sn[e] = __shfl_sync(FULL, s2[e & 1], from) * g;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + 4 * u;
            const bool live = h < a.heads && (h < a.Hq || slot >= 0);
            const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
            const __nv_bfloat16 *w = is_q ? a.wq : a.wk;
            uint4 y0, y1;
            float x[8], y[8];
            if (live && !is_v) {
                unpack8(w0[u], x);
                unpack8(w1[u], y);
            }
            if (a.wq != nullptr || a.wk != nullptr) {  // uniform: the sum below is a warp's
                float ss = 0.f;
                if (live && !is_v)
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(FULL, ss, o);
                if (live && !is_v && w != nullptr) {
                    const float r = rsqrtf(fmaf(ss, 1.f / ROPE_D, a.eps));
                    float g0[8], g1[8];
                    unpack8(__ldg(reinterpret_cast<const uint4 *>(w + c0)), g0);
                    unpack8(__ldg(reinterpret_cast<const uint4 *>(w + c1)), g1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] *= r * g0[e];
                        y[e] *= r * g1[e];
                    }
                }
            }
            if (!live) continue;
            if (is_v) {
                y0 = w0[u];
                y1 = w1[u];
            } else {
                if (rot) {
                    if (INTER) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p0 = x[2 * e], p1 = x[2 * e + 1], q0 = y[2 * e], q1 = y[2 * e + 1];
                            x[2 * e] = fmaf(p0, cs[e], -p1 * sn[e]);
                            x[2 * e + 1] = fmaf(p1, cs[e], p0 * sn[e]);
                            y[2 * e] = fmaf(q0, cs[e + 4], -q1 * sn[e + 4]);
                            y[2 * e + 1] = fmaf(q1, cs[e + 4], q0 * sn[e + 4]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float p0 = x[e], p1 = y[e];
                            x[e] = fmaf(p0, cs[e], -p1 * sn[e]);
                            y[e] = fmaf(p1, cs[e], p0 * sn[e]);
                        }
                    }
                }
                y0 = pack8(x);
                y1 = pack8(y);
            }
            __nv_bfloat16 *dst;
            if (is_q) {
                dst = a.out_q + token * a.out_q_stride + (int64_t)h * ROPE_D;
            } else if (a.k_cache == nullptr) {
                dst = a.out_k + token * a.out_k_stride + (int64_t)(h - a.Hq) * ROPE_D;
            } else if (!is_v) {
                dst = a.k_cache + (slot * a.Hkv + (h - a.Hq)) * ROPE_D;
            } else {
                dst = a.v_cache + (slot * a.Hkv + (h - a.Hq - a.Hkv)) * ROPE_D;
            }
            *reinterpret_cast<uint4 *>(dst + c0) = y0;
            *reinterpret_cast<uint4 *>(dst + c1) = y1;
        }
    }
}

template <bool INTER, int U>
pa_status launch_rope(RopeArgs &a, int sms, cudaStream_t stream) {
    a.parts = (a.heads + 4 * U - 1) / (4 * U);
    const int64_t units = (int64_t)a.tokens * a.parts, warps = ROPE_THREADS / 32;
    const int64_t grid = std::min<int64_t>((units + warps - 1) / warps, 8LL * sms);
    return launch_pdl(rope_kernel<INTER, U>, dim3((unsigned)grid), dim3(ROPE_THREADS), 0, stream, "rope_kernel", a);
}

// Checks and launches what the two entry points share.
pa_status run_rope(RopeArgs &a, int32_t head_dim, int32_t interleaved, pa_stream_t stream) {
    if (!a.q || !a.k || !a.out_q || !a.positions || !a.freqs) return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (a.Hq <= 0 || a.Hkv <= 0 || head_dim <= 0) return fail(PA_ERR_INVALID_ARG, "bad head shape");
    if (head_dim != ROPE_D) return fail(PA_ERR_UNSUPPORTED, "head_dim %d (only 128)", head_dim);
    if (a.Hq > (1 << 20) || a.Hkv > (1 << 20)) return fail(PA_ERR_UNSUPPORTED, "too many heads");
    if (a.rotary < 16 || a.rotary > ROPE_D || a.rotary % 16)
        return fail(PA_ERR_UNSUPPORTED, "rotary_dim %d (a multiple of 16 up to 128)", a.rotary);
    if (interleaved != 0 && interleaved != 1) return fail(PA_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!(a.eps >= 0.f)) return fail(PA_ERR_INVALID_ARG, "eps must not be negative");
    const int64_t qrow = (int64_t)a.Hq * ROPE_D, krow = (int64_t)a.Hkv * ROPE_D;
    if (a.q_stride < qrow || a.out_q_stride < qrow || a.k_stride < krow || (a.v && a.v_stride < krow) ||
        (a.out_k && a.out_k_stride < krow))
        return fail(PA_ERR_INVALID_ARG, "row stride smaller than a token's heads");
    if (a.q_stride % 8 || a.out_q_stride % 8 || a.k_stride % 8 || (a.v && a.v_stride % 8) ||
        (a.out_k && a.out_k_stride % 8))
        return fail(PA_ERR_INVALID_ARG, "row strides must be multiples of 8 elements");
    if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.out_q) || !aligned16(a.out_k) ||
        !aligned16(a.k_cache) || !aligned16(a.v_cache) || !aligned16(a.wq) || !aligned16(a.wk))
        return fail(PA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(a.freqs) & 7u) return fail(PA_ERR_INVALID_ARG, "freqs must be 8-byte aligned");
    if ((int64_t)a.tokens * ((a.heads + 3) / 4) > 0x7fffffff) return fail(PA_ERR_INVALID_ARG, "num_tokens too large");
    const int sms = sm_count();
    if (sms <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    a.err = device_error_ptr();
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return interleaved ? launch_rope<true, 4>(a, sms, s) : launch_rope<false, 4>(a, sms, s);
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_rope_frequencies(uint64_t *freqs, float *gain, int32_t rotary_dim, double theta, int32_t scaling,
                              double factor, double original_context, double beta_fast, double beta_slow) {
    using namespace pa;
    if (!freqs || !gain) return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (rotary_dim < 16 || rotary_dim > ROPE_D || rotary_dim % 16)
        return fail(PA_ERR_UNSUPPORTED, "rotary_dim %d (a multiple of 16 up to 128)", rotary_dim);
    if (!(theta > 1.0) || !isfinite(theta)) return fail(PA_ERR_INVALID_ARG, "theta must be above 1");
    if (scaling < PA_ROPE_PLAIN || scaling > PA_ROPE_YARN) return fail(PA_ERR_INVALID_ARG, "unknown scaling %d", scaling);
    if (scaling != PA_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor)))
        return fail(PA_ERR_INVALID_ARG, "factor must be at least 1");
    const double r = rotary_dim, two_pi = 6.283185307179586476925286766559;
    double lo = 0, hi = 0;
    if (scaling == PA_ROPE_YARN) {
        if (!(original_context > 0) || !(beta_slow > 0) || !(beta_fast >= beta_slow) || !isfinite(original_context) ||
            !isfinite(beta_fast))
            return fail(PA_ERR_INVALID_ARG, "original_context and beta_fast >= beta_slow must be positive");
        lo = std::max(floor(r * log(original_context / (beta_fast * two_pi)) / (2 * log(theta))), 0.0);
        hi = std::min(ceil(r * log(original_context / (beta_slow * two_pi)) / (2 * log(theta))), r - 1);
    }
    if (scaling == PA_ROPE_NTK) theta *= pow(factor, r / (r - 2));
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(theta, -2.0 * i / r);
        if (scaling == PA_ROPE_LINEAR) f /= factor;
        if (scaling == PA_ROPE_YARN) {
            const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
            f = f * (1 - ramp) + f / factor * ramp;
        }
        freqs[i] = static_cast<uint64_t>(f / two_pi * 18446744073709551616.0);  // f <= 1: below 2^62
    }
    *gain = static_cast<float>(scaling == PA_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0);
    return PA_OK;
}

pa_status pa_rope(void *out_q, int64_t out_q_row_stride, void *out_k, int64_t out_k_row_stride, const void *q,
                  int64_t q_row_stride, const void *key, int64_t key_row_stride, const int32_t *positions,
                  const uint64_t *freqs, int32_t rotary_dim, int32_t interleaved, float gain, const void *q_norm,
                  const void *k_norm, float eps, int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                  int32_t head_dim, pa_stream_t stream) {
    using namespace pa;
    if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if (num_tokens == 0) return PA_OK;
    if (!out_k) return fail(PA_ERR_INVALID_ARG, "null pointer");
    RopeArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(key);
    a.q_stride = q_row_stride;
    a.k_stride = key_row_stride;
    a.out_q = static_cast<__nv_bfloat16 *>(out_q);
    a.out_k = static_cast<__nv_bfloat16 *>(out_k);
    a.out_q_stride = out_q_row_stride;
    a.out_k_stride = out_k_row_stride;
    a.positions = positions;
    a.freqs = reinterpret_cast<const unsigned long long *>(freqs);
    a.wq = static_cast<const __nv_bfloat16 *>(q_norm);
    a.wk = static_cast<const __nv_bfloat16 *>(k_norm);
    a.gain = gain;
    a.eps = eps;
    a.tokens = num_tokens;
    a.Hq = num_q_heads;
    a.Hkv = num_kv_heads;
    a.heads = num_q_heads + num_kv_heads;
    a.rotary = rotary_dim;
    return run_rope(a, head_dim, interleaved, stream);
}

pa_status pa_rope_store_kvcache(void *out_q, int64_t out_q_row_stride, const void *q, int64_t q_row_stride,
                                const void *key, int64_t key_row_stride, const void *value, int64_t value_row_stride,
                                const int32_t *positions, const uint64_t *freqs, int32_t rotary_dim,
                                int32_t interleaved, float gain, const void *q_norm, const void *k_norm, float eps,
                                void *k_cache, void *v_cache, const int32_t *slot_mapping, int32_t num_tokens,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int64_t num_slots,
                                pa_stream_t stream) {
    using namespace pa;
    if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if (num_tokens == 0) return PA_OK;
    if (!value || !k_cache || !v_cache || !slot_mapping) return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (num_slots <= 0) return fail(PA_ERR_INVALID_ARG, "num_slots <= 0");
    RopeArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(key);
    a.v = static_cast<const __nv_bfloat16 *>(value);
    a.q_stride = q_row_stride;
    a.k_stride = key_row_stride;
    a.v_stride = value_row_stride;
    a.out_q = static_cast<__nv_bfloat16 *>(out_q);
    a.out_q_stride = out_q_row_stride;
    a.k_cache = static_cast<__nv_bfloat16 *>(k_cache);
    a.v_cache = static_cast<__nv_bfloat16 *>(v_cache);
    a.slots = slot_mapping;
    a.num_slots = num_slots;
    a.positions = positions;
    a.freqs = reinterpret_cast<const unsigned long long *>(freqs);
    a.wq = static_cast<const __nv_bfloat16 *>(q_norm);
    a.wk = static_cast<const __nv_bfloat16 *>(k_norm);
    a.gain = gain;
    a.eps = eps;
    a.tokens = num_tokens;
    a.Hq = num_q_heads;
    a.Hkv = num_kv_heads;
    a.heads = num_q_heads + 2 * num_kv_heads;
    a.rotary = rotary_dim;
    return run_rope(a, head_dim, interleaved, stream);
}

}  // extern "C"
