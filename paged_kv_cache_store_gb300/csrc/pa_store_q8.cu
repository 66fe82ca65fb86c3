// pa_store_q8.cu -- writing rows into an 8-bit KV pool, and reading them back.
//
// The pool is head-major, [num_blocks, Hkv, block_size, 128] codes and
// [num_blocks, Hkv, block_size] scale bytes: the keys of one (block, head),
// which attention streams, are contiguous.  (Streaming 32-key K and V tiles
// of scattered blocks by TMA measured 7.1-7.3 TB/s this way and 4.7-4.8 TB/s
// from 128-byte rows a token apart, [num_blocks, block_size, Hkv, 128].)
//
// Store: a half-warp takes one (token, K or V, head) row: 16 lanes x 16 bytes
// of bf16, the row's largest magnitude by four shuffles, then 8 codes a lane.
// Load: the same units the other way.  Both are pure streams (store: 256 bytes
// read and 129 written a row; load: 129 and 256), so a half-warp keeps UNITS
// rows' loads in flight before it works on the first.
#include <algorithm>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int Q8_THREADS = 256;
constexpr int UNITS = 4;  // rows in flight per half-warp

struct Q8Rows {
    uint4 *key, *value;             // the bf16 rows (store: read, load: written)
    int64_t key16, value16;         // 16-byte units between tokens
    uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
    const int32_t *slots;
    uint32_t num_tokens, hkv, block;
    int64_t num_slots;
    DevError *err;
};

// Row r of the call: token, K or V, head (heads innermost, as the rows lie).
struct Unit {
    uint4 *rows;             // the unit's 256 bytes of bf16
    uint8_t *codes, *scale;  // its codes and scale byte (null: nothing to read or write)
    bool live;
};

__device__ __forceinline__ Unit unit_of(const Q8Rows &a, uint64_t r, uint64_t n, int lane16) {
    Unit u;
    u.live = r < n;
    if (!u.live) r = 0;
    const uint32_t per = 2 * a.hkv;
    const uint32_t token = n <= 0xffffffffull ? (uint32_t)r / per : (uint32_t)(r / per);
    const uint32_t rest = (uint32_t)(r - (uint64_t)token * per);
    const bool is_v = rest >= a.hkv;
    const uint32_t head = is_v ? rest - a.hkv : rest;
    u.rows = (is_v ? a.value + token * a.value16 : a.key + token * a.key16) + head * (Q8_D / 8) + lane16;
    u.codes = u.scale = nullptr;
    const int32_t slot = __ldg(a.slots + token);
    if (slot >= 0 && slot < a.num_slots) {
        const uint32_t blk = (uint32_t)slot / a.block, off = (uint32_t)slot - blk * a.block;
        const int64_t row = ((int64_t)blk * a.hkv + head) * a.block + off;
        u.codes = (is_v ? a.v_codes : a.k_codes) + row * Q8_D + 8 * lane16;
        u.scale = (is_v ? a.v_scales : a.k_scales) + row;
    } else if (slot >= 0 && u.live && rest == 0 && lane16 == 0) {
        record_error(a.err, PA_DEV_BAD_SLOT, token);
    }
    return u;
}

__device__ __forceinline__ uint4 ld_stream16(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// max of packed bf16 magnitudes that keeps a NaN.
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int FMT>
__global__ void __launch_bounds__(Q8_THREADS) store_kvcache_q8_kernel(const Q8Rows a) {
    pdl_wait_then_release();
    const int lane16 = threadIdx.x & 15;
    const uint64_t n = 2ull * a.num_tokens * a.hkv;
    const uint64_t hw = ((uint64_t)blockIdx.x * Q8_THREADS + threadIdx.x) >> 4;
    const uint64_t nhw = (uint64_t)gridDim.x * (Q8_THREADS / 16);
    // Both halves of a warp run the same trips (the shuffles need them).
    for (uint64_t r0 = hw; (r0 & ~1ull) < n; r0 += nhw * UNITS) {
        Unit u[UNITS];
        uint4 v[UNITS];
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            u[i] = unit_of(a, r0 + i * nhw, n, lane16);
            v[i] = make_uint4(0, 0, 0, 0);
            if (u[i].live && u[i].codes) v[i] = ld_stream16(u[i].rows);
        }
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t mx = w[0] & 0x7fff7fffu;
#pragma unroll
            for (int j = 1; j < 4; ++j) mx = max_nan_bf16x2(mx, w[j] & 0x7fff7fffu);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) mx = max_nan_bf16x2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // Magnitudes order as their bits (a NaN above all).
            const uint32_t amax = max(mx & 0xffffu, mx >> 16);
            const bool finite = amax < 0x7f80u;
            const int e = q8_exponent<FMT>(amax);
            const float inv = __uint_as_float((uint32_t)(127 - (finite ? e : 0)) << 23);
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = finite ? bf16lo(w[j]) * inv : 0.f;
                f[2 * j + 1] = finite ? bf16hi(w[j]) * inv : 0.f;
            }
            if (u[i].live && u[i].codes) {
                uint2 c;
                c.x = q8_encode4<FMT>(f[0], f[1], f[2], f[3]);
                c.y = q8_encode4<FMT>(f[4], f[5], f[6], f[7]);
                *reinterpret_cast<uint2 *>(u[i].codes) = c;
                if (lane16 == 0) *u[i].scale = (uint8_t)(finite ? e + 127 : 255);
            }
        }
    }
}

template <int FMT>
__global__ void __launch_bounds__(Q8_THREADS) load_kvcache_q8_kernel(const Q8Rows a) {
    pdl_wait_then_release();
    const int lane16 = threadIdx.x & 15;
    const uint64_t n = 2ull * a.num_tokens * a.hkv;
    const uint64_t hw = ((uint64_t)blockIdx.x * Q8_THREADS + threadIdx.x) >> 4;
    const uint64_t nhw = (uint64_t)gridDim.x * (Q8_THREADS / 16);
    for (uint64_t r0 = hw; r0 < n; r0 += nhw * UNITS) {
        Unit u[UNITS];
        uint2 c[UNITS];
        uint32_t s[UNITS];
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            u[i] = unit_of(a, r0 + i * nhw, n, lane16);
            c[i] = make_uint2(0, 0);
            s[i] = 127;
            if (u[i].live && u[i].codes) {
                c[i] = __ldg(reinterpret_cast<const uint2 *>(u[i].codes));
                s[i] = __ldg(u[i].scale);
            }
        }
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            if (!u[i].live) continue;
            uint4 o = make_uint4(0, 0, 0, 0);  // a negative (or bad) slot reads as zeros
            if (u[i].codes) {
                const float sc = q8_scale(s[i]);
                uint32_t h[4];
                q8_to_f16<FMT>(c[i].x, h[0], h[1]);
                q8_to_f16<FMT>(c[i].y, h[2], h[3]);
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
                    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * sc, f.y * sc);
                    w[j] = *reinterpret_cast<const uint32_t *>(&b);
                }
                o = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *u[i].rows = o;
        }
    }
}

pa_status launch_rows(const Q8Rows &a, int32_t format, bool store, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    // A half-warp per row and step; at most 8 CTAs of 16 half-warps per SM.
    const int64_t rows = 2LL * a.num_tokens * a.hkv, per = Q8_THREADS / 16;
    const dim3 grid((unsigned)std::min<int64_t>((rows + per - 1) / per, 8LL * sms)), block(Q8_THREADS);
    if (store)
        return format == PA_Q8_E4M3
                   ? launch_pdl(store_kvcache_q8_kernel<PA_Q8_E4M3>, grid, block, 0, stream, "store_kvcache_q8_kernel", a)
                   : launch_pdl(store_kvcache_q8_kernel<PA_Q8_INT8>, grid, block, 0, stream, "store_kvcache_q8_kernel", a);
    return format == PA_Q8_E4M3
               ? launch_pdl(load_kvcache_q8_kernel<PA_Q8_E4M3>, grid, block, 0, stream, "load_kvcache_q8_kernel", a)
               : launch_pdl(load_kvcache_q8_kernel<PA_Q8_INT8>, grid, block, 0, stream, "load_kvcache_q8_kernel", a);
}

pa_status rows_impl(const void *key, int64_t key_row_stride, const void *value, int64_t value_row_stride,
                    const void *k_cache, const void *v_cache, const void *k_scale, const void *v_scale,
                    const int32_t *slot_mapping, int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                    int32_t block_size, int32_t num_blocks, int32_t format, bool store, pa_stream_t stream) {
    if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !k_scale || !v_scale || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    const pa_status st = q8_check_pool(format, num_kv_heads, head_dim, block_size, num_blocks);
    if (st != PA_OK) return st;
    const int64_t row = (int64_t)num_kv_heads * head_dim;
    if (key_row_stride < row || value_row_stride < row)
        return fail(PA_ERR_INVALID_ARG, "row stride smaller than num_kv_heads*head_dim");
    if (key_row_stride % 8 || value_row_stride % 8)
        return fail(PA_ERR_INVALID_ARG, "row strides must be multiples of 8 elements");
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) ||
        !aligned16(v_scale))
        return fail(PA_ERR_INVALID_ARG, "row, cache and scale pointers must be 16-byte aligned");
    Q8Rows a = {};
    a.key = static_cast<uint4 *>(const_cast<void *>(key));
    a.value = static_cast<uint4 *>(const_cast<void *>(value));
    a.key16 = key_row_stride / 8;
    a.value16 = value_row_stride / 8;
    a.k_codes = static_cast<uint8_t *>(const_cast<void *>(k_cache));
    a.v_codes = static_cast<uint8_t *>(const_cast<void *>(v_cache));
    a.k_scales = static_cast<uint8_t *>(const_cast<void *>(k_scale));
    a.v_scales = static_cast<uint8_t *>(const_cast<void *>(v_scale));
    a.slots = slot_mapping;
    a.num_tokens = (uint32_t)num_tokens;
    a.hkv = (uint32_t)num_kv_heads;
    a.block = (uint32_t)block_size;
    a.num_slots = (int64_t)num_blocks * block_size;
    a.err = device_error_ptr();
    return launch_rows(a, format, store, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_store_kvcache_q8(const void *key, int64_t key_row_stride, const void *value, int64_t value_row_stride,
                              void *k_cache, void *v_cache, void *k_scale, void *v_scale,
                              const int32_t *slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t format,
                              pa_stream_t stream) {
    return pa::rows_impl(key, key_row_stride, value, value_row_stride, k_cache, v_cache, k_scale, v_scale,
                         slot_mapping, num_tokens, num_kv_heads, head_dim, block_size, num_blocks, format, true,
                         stream);
}

pa_status pa_load_kvcache_q8(void *key, int64_t key_row_stride, void *value, int64_t value_row_stride,
                             const void *k_cache, const void *v_cache, const void *k_scale, const void *v_scale,
                             const int32_t *slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                             int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t format,
                             pa_stream_t stream) {
    return pa::rows_impl(key, key_row_stride, value, value_row_stride, k_cache, v_cache, k_scale, v_scale,
                         slot_mapping, num_tokens, num_kv_heads, head_dim, block_size, num_blocks, format, false,
                         stream);
}

}  // extern "C"
