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
// The angle: f_i is a fraction of 2^64, rounded to the nearest, and p * f_i is taken
// modulo 2^64, so the turns are off by |p| 2^-65 (2^-34 at the farthest 32-bit
// position); the signed result is rounded once to fp32 (an angle error of at most
// 2^-25 pi) before sincospif.  The product in fp32 would be off by 4e-3 at position 10^5
// and by 3e-2 at 10^6.
//
// Layout: eight lanes per head, two 16-byte chunks a lane, chosen so that both
// halves of a pair are in one lane: chunks 8l and R/2 + 8l of the rotated part
// (split halves), 16l and 16l + 8 otherwise.  A warp's four lane groups take four
// heads and share the token's 64 angles: each lane evaluates two and gets its
// eight by shuffles.
//
// What bounds it: a step's tokens the launch (64 tokens of 32 + 8 + 8 heads 2.9 us); a
// prefill HBM and the issue slots (16384 tokens, norm, store: 73 us, 403 MB, 5.5 TB/s
// or 82 % of the copy's rate, 39 % of the issue slots), as the rows go to scattered slots.
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
    int32_t tokens, Hq, Hkv, groups;       // groups of four heads of a token: of q, k, and (store) v
    int32_t rotary, span, parts;           // groups of a unit, units of a token
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

// Two fp32 at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// A unit is one token and `span` of its groups of four heads: those of q, then of k,
// then (store) of v.  A head's output is X P + X' Q and Y R + Y' S, times the norm's
// factor, with X and Y the lane's two chunks, X' and Y' the pairs' other halves
// (the other chunk, or the neighbours), and P, Q, R, S the angles' cosines and sines
// times gain and weight: made once per token for all heads of q, and of k.  U groups
// are under way at a time.
template <bool INTER, bool NORM, int U>
__global__ void __launch_bounds__(ROPE_THREADS, 2) rope_kernel(const __grid_constant__ RopeArgs a) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31, l = lane & 7, grp = lane >> 3;
    const bool rot = 16 * l < a.rotary;
    const int c0 = (INTER || !rot) ? 16 * l : 8 * l;
    const int c1 = (INTER || !rot) ? 16 * l + 8 : a.rotary / 2 + 8 * l;
    const uint32_t nunits = (uint32_t)a.tokens * (uint32_t)a.parts;
    const uint32_t wstride = gridDim.x * (ROPE_THREADS / 32);
    const int gq = (a.Hq + 3) >> 2, gk = (a.Hkv + 3) >> 2;
    // The two pairs whose angle this lane evaluates.
    unsigned long long f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) f[e] = rot ? __ldg(a.freqs + 8 * l + 2 * grp + e) : 0ull;
    for (uint32_t unit = blockIdx.x * (ROPE_THREADS / 32) + (threadIdx.x >> 5); unit < nunits; unit += wstride) {
        const uint32_t token = unit / (uint32_t)a.parts, part = unit - token * (uint32_t)a.parts;
        const int g0 = (int)part * a.span, g1 = min(g0 + a.span, a.groups);
        const long long pos = __ldg(a.positions + token);
        int64_t slot = 0;
        if (a.k_cache != nullptr) {
            slot = __ldg(a.slots + token);
            if (slot >= a.num_slots) {
                if (g0 == 0 && lane == 0) record_error(a.err, PA_DEV_BAD_SLOT, token);
                slot = -1;
            }
        }
        float cs[8], sn[8];
        {
            float c2[2], s2[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const long long turns = (long long)((unsigned long long)pos * f[e]);  // in 2^-64, -1/2 .. 1/2
                sincospif((float)turns * 0x1p-63f, &s2[e], &c2[e]);
            }
            const float g = rot ? a.gain : 1.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int from = (e >> 1) * 8 + l;
                cs[e] = __shfl_sync(FULL, c2[e & 1], from) * g;
                sn[e] = __shfl_sync(FULL, s2[e & 1], from) * g;
            }
        }
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {  // q, k
            const int b0 = kind ? gq : 0, b1 = kind ? gq + gk : gq, heads = kind ? a.Hkv : a.Hq;
            const int from = max(g0, b0) - b0, to = min(g1, b1) - b0;
            if (from >= to || (kind && slot < 0)) continue;
            const __nv_bfloat16 *src = kind ? a.k + token * a.k_stride : a.q + token * a.q_stride;
            __nv_bfloat16 *dst = !kind                     ? a.out_q + token * a.out_q_stride
                                 : a.k_cache == nullptr ? a.out_k + token * a.out_k_stride
                                                        : a.k_cache + slot * a.Hkv * ROPE_D;
            const __nv_bfloat16 *weight = kind ? a.wk : a.wq;
            const bool norm = NORM && weight != nullptr;
            float2 P[4], Q[4], R[4], S[4];
            {
                float g0w[8], g1w[8];
                if (norm) {
                    unpack8(__ldg(reinterpret_cast<const uint4 *>(weight + c0)), g0w);
                    unpack8(__ldg(reinterpret_cast<const uint4 *>(weight + c1)), g1w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float w0 = norm ? g0w[2 * e] : 1.f, w1 = norm ? g0w[2 * e + 1] : 1.f;
                    const float v0 = norm ? g1w[2 * e] : 1.f, v1 = norm ? g1w[2 * e + 1] : 1.f;
                    if (!rot) {
                        P[e] = make_float2(w0, w1);
                        R[e] = make_float2(v0, v1);
                        Q[e] = S[e] = make_float2(0.f, 0.f);
                    } else if (INTER) {  // pairs e of the first chunk, e + 4 of the second
                        P[e] = make_float2(w0 * cs[e], w1 * cs[e]);
                        Q[e] = make_float2(-w1 * sn[e], w0 * sn[e]);
                        R[e] = make_float2(v0 * cs[e + 4], v1 * cs[e + 4]);
                        S[e] = make_float2(-v1 * sn[e + 4], v0 * sn[e + 4]);
                    } else {
                        P[e] = make_float2(w0 * cs[2 * e], w1 * cs[2 * e + 1]);
                        Q[e] = make_float2(-v0 * sn[2 * e], -v1 * sn[2 * e + 1]);
                        R[e] = make_float2(v0 * cs[2 * e], v1 * cs[2 * e + 1]);
                        S[e] = make_float2(w0 * sn[2 * e], w1 * sn[2 * e + 1]);
                    }
                }
            }
#pragma unroll 1
            for (int g = from; g < to; g += U) {
                uint4 w0[U], w1[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = 4 * (g + u) + grp;
                    if (g + u < to && h < heads) {
                        w0[u] = ld_row16(src + h * ROPE_D + c0);
                        w1[u] = ld_row16(src + h * ROPE_D + c1);
                    } else {
                        w0[u] = w1[u] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int h = 4 * (g + u) + grp;
                    float x[8], y[8];
                    unpack8(w0[u], x);
                    unpack8(w1[u], y);
                    float r = 1.f;
                    if (NORM && norm) {
                        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float2 X = make_float2(x[e], x[e + 1]), Y = make_float2(y[e], y[e + 1]);
                            ss = fma2(X, X, fma2(Y, Y, ss));
                        }
                        float t = ss.x + ss.y;
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) t += __shfl_xor_sync(FULL, t, o);
                        r = rsqrtf(fmaf(t, 1.f / ROPE_D, a.eps));
                    }
                    if (g + u >= to || h >= heads) continue;
                    if (rot || (NORM && norm)) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 X = make_float2(x[2 * e], x[2 * e + 1]), Y = make_float2(y[2 * e], y[2 * e + 1]);
                            float2 X1 = mul2(X, P[e]), Y1 = mul2(Y, R[e]);
                            if (rot) {
                                X1 = fma2(INTER ? make_float2(X.y, X.x) : Y, Q[e], X1);
                                Y1 = fma2(INTER ? make_float2(Y.y, Y.x) : X, S[e], Y1);
                            }
                            if (NORM) {
                                X1 = mul2(X1, make_float2(r, r));
                                Y1 = mul2(Y1, make_float2(r, r));
                            }
                            x[2 * e] = X1.x;
                            x[2 * e + 1] = X1.y;
                            y[2 * e] = Y1.x;
                            y[2 * e + 1] = Y1.y;
                        }
                        w0[u] = pack8(x);
                        w1[u] = pack8(y);
                    }
                    *reinterpret_cast<uint4 *>(dst + h * ROPE_D + c0) = w0[u];
                    *reinterpret_cast<uint4 *>(dst + h * ROPE_D + c1) = w1[u];
                }
            }
        }
        // v: copied
        if (a.v == nullptr || slot < 0) continue;
        const __nv_bfloat16 *src = a.v + token * a.v_stride;
        __nv_bfloat16 *dst = a.v_cache + slot * a.Hkv * ROPE_D;
        const int from = max(g0, gq + gk) - (gq + gk), to = g1 - (gq + gk);
        for (int h = 4 * from + grp; h < min(4 * to, a.Hkv); h += 4) {
            const uint4 t0 = ld_row16(src + h * ROPE_D + 16 * l), t1 = ld_row16(src + h * ROPE_D + 16 * l + 8);
            *reinterpret_cast<uint4 *>(dst + h * ROPE_D + 16 * l) = t0;
            *reinterpret_cast<uint4 *>(dst + h * ROPE_D + 16 * l + 8) = t1;
        }
    }
}

// Numbers of some 105 bits, the sum of two doubles: a frequency's 64 bits are more than one
// holds.  (A sum's and a product's rounding error is a double, which fma and differences
// give exactly.)
struct Wide {
    double hi, lo;
};
Wide norm(double a, double b) {  // |a| >= |b|
    const double s = a + b;
    return {s, b - (s - a)};
}
Wide add(Wide a, Wide b) {
    const double s = a.hi + b.hi, t = s - a.hi;
    return norm(s, (a.hi - (s - t)) + (b.hi - t) + a.lo + b.lo);
}
Wide mul(Wide a, Wide b) {
    const double p = a.hi * b.hi;
    return norm(p, fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Wide div(Wide a, double b) {
    const double q = a.hi / b, rest = fma(-q, b, a.hi) + a.lo;
    return norm(q, rest / b);
}
// a^(-1/n): the root of a x^n = 1, by Newton's steps from double's.
Wide inverse_root(double a, int n) {
    Wide x = {pow(a, -1.0 / n), 0.0};
    for (int step = 0; step < 2; ++step) {
        Wide y = {-a, 0.0};  // to -a x^n, from the large end, so that nothing underflows
        for (int i = 0; i < n; ++i) y = mul(y, x);
        x = add(x, div(mul(x, add({1.0, 0.0}, y)), n));
    }
    return x;
}

template <bool INTER, bool NORM, int U>
pa_status launch_rope(const RopeArgs &a, int sms, cudaStream_t stream) {
    const int64_t units = (int64_t)a.tokens * a.parts, warps = ROPE_THREADS / 32;
    const int64_t grid = std::min<int64_t>((units + warps - 1) / warps, 2LL * sms);
    return launch_pdl(rope_kernel<INTER, NORM, U>, dim3((unsigned)grid), dim3(ROPE_THREADS), 0, stream, "rope_kernel", a);
}

template <bool INTER, bool NORM>
pa_status launch_rope(RopeArgs &a, int sms, cudaStream_t stream) {
    // Units of a whole token, its angles evaluated once, while there are warps enough
    // for the GPU (16 per SM); smaller ones, down to one group of heads, below that.
    // Whole tokens take four groups of heads at a time (16384 tokens 72.8 us, two at
    // a time 74.2), parts of them two (512 tokens 5.4 us, four at a time 6.5).
    a.span = (int)std::max<int64_t>(1, std::min<int64_t>(a.groups, (int64_t)a.tokens * a.groups / (16LL * sms)));
    a.parts = (a.groups + a.span - 1) / a.span;
    return a.parts == 1 ? launch_rope<INTER, NORM, 4>(a, sms, stream) : launch_rope<INTER, NORM, 2>(a, sms, stream);
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
    if ((int64_t)a.tokens * a.groups > 0x7fffffff) return fail(PA_ERR_INVALID_ARG, "num_tokens too large");
    const int sms = sm_count();
    if (sms <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    a.err = device_error_ptr();
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a.wq || a.wk) return interleaved ? launch_rope<true, true>(a, sms, s) : launch_rope<false, true>(a, sms, s);
    return interleaved ? launch_rope<true, false>(a, sms, s) : launch_rope<false, false>(a, sms, s);
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
    // f_i is the i-th power of theta^(-2/R), for ntk times s^(-2/(R-2)).
    Wide step = inverse_root(theta, rotary_dim / 2);
    if (scaling == PA_ROPE_NTK) step = mul(step, inverse_root(factor, rotary_dim / 2 - 1));
    Wide f = {0.15915494309189535, -9.839338337591243e-18};  // 1 / (2 pi)
    for (int i = 0; i < rotary_dim / 2; ++i, f = mul(f, step)) {
        Wide x = f;
        if (scaling == PA_ROPE_LINEAR) x = div(f, factor);
        if (scaling == PA_ROPE_YARN) {  // f (1 - ramp) + f / s * ramp
            if (i >= hi) {
                x = i > lo ? div(f, factor) : f;
            } else if (i > lo) {
                const Wide short_part = div(mul(f, {hi - i, 0.0}), hi - lo);
                x = add(short_part, div(div(mul(f, {i - lo, 0.0}), hi - lo), factor));
            }
        }
        const double whole = rint(x.hi * 0x1p64);  // (f <= 1: below 2^62)
        freqs[i] = static_cast<uint64_t>(whole) + static_cast<uint64_t>(llrint((x.hi * 0x1p64 - whole) + x.lo * 0x1p64));
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
    a.groups = (num_q_heads + 3) / 4 + (num_kv_heads + 3) / 4;
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
    a.groups = (num_q_heads + 3) / 4 + 2 * ((num_kv_heads + 3) / 4);
    a.rotary = rotary_dim;
    return run_rope(a, head_dim, interleaved, stream);
}

}  // extern "C"
