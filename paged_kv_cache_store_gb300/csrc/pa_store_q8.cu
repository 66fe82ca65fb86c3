// pa_store_q8.cu -- writing rows into an 8-bit KV pool, and reading them back.
//
// The pool is head-major, [num_blocks, Hkv, block_size, 128] codes and
// [num_blocks, Hkv, block_size] scale bytes: the keys of one (block, head),
// which attention streams, are contiguous.  (Streaming 32-key K and V tiles
// of scattered blocks by TMA measured 7.1-7.3 TB/s this way and 4.7-4.8 TB/s
// from 128-byte rows a token apart, [num_blocks, block_size, Hkv, 128].)
//
// Store: eight lanes take up to H heads' rows of one (token, K or V): 2 x 16
// bytes of bf16 a lane and row (dims 8i.. and 64 + 8i..), the row's largest
// magnitude by three shuffles, then 16 codes a lane.  Load: the same the other
// way.  Both are pure streams (store: 256 bytes read and 129 written a row;
// load: 129 and 256) that would be bound by instructions if each row found its
// own slot, block and offset (three divisions; 2.8 TB/s): the unit's rows share
// them, and the next unit's slot travels while this one's rows do.  H is 2 in the
// store (six CTAs an SM; 16384 tokens 19.1 us, with H = 4 and four CTAs 19.5) and
// 4 in the load (16384 tokens 14.7 us, with 2 15.8), or less in small calls.
#include <algorithm>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int Q8_THREADS = 256;
constexpr int LANES = 8;                        // of a unit
constexpr int UNITS = Q8_THREADS / LANES;       // of a CTA

struct Q8Rows {
    uint4 *key, *value;             // the bf16 rows (store: read, load: written)
    int64_t key16, value16;         // 16-byte units between tokens
    uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
    const int32_t *slots;
    uint32_t num_tokens, hkv, block, groups;  // groups of H heads
    int64_t num_slots;
    DevError *err;
};

// Up to H heads' rows of a token's K or V.
struct Unit {
    uint4 *rows;             // this lane's first 16 bytes of the first row
    uint8_t *codes, *scale;  // its first 8 codes, and the row's scale byte
    uint32_t n;              // rows
    bool live;               // a slot of the pool
};

// Unit u: token, K or V, group of heads (innermost).
__device__ __forceinline__ uint32_t token_of(const Q8Rows &a, uint64_t u) {
    const uint32_t per = 2 * a.groups;
    return u <= 0xffffffffull ? (uint32_t)u / per : (uint32_t)(u / per);
}
template <uint32_t H>
__device__ __forceinline__ Unit unit_of(const Q8Rows &a, uint64_t u, uint32_t token, int32_t slot, int lane) {
    const uint32_t rest = (uint32_t)(u - (uint64_t)token * (2 * a.groups));
    const bool is_v = rest >= a.groups;
    const uint32_t head = (is_v ? rest - a.groups : rest) * H;
    Unit r;
    r.n = min(H, a.hkv - head);
    r.rows = (is_v ? a.value + token * a.value16 : a.key + token * a.key16) + head * (Q8_D / 8) + lane;
    r.live = slot >= 0 && slot < a.num_slots;
    if (slot >= 0 && !r.live && rest == 0 && lane == 0) record_error(a.err, PA_DEV_BAD_SLOT, token);
    const uint32_t at = r.live ? (uint32_t)slot : 0u, blk = at / a.block, off = at - blk * a.block;
    const int64_t row = ((int64_t)blk * a.hkv + head) * a.block + off;
    r.codes = (is_v ? a.v_codes : a.k_codes) + row * Q8_D + 8 * lane;
    r.scale = (is_v ? a.v_scales : a.k_scales) + row;
    return r;
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

template <int FMT, uint32_t H>
__global__ void __launch_bounds__(Q8_THREADS, 6) store_kvcache_q8_kernel(const Q8Rows a) {
    pdl_wait_then_release();
    const int lane = threadIdx.x % LANES;
    const unsigned group = 0xffu << (threadIdx.x & 24);  // this unit's lanes
    const uint64_t n = 2ull * a.num_tokens * a.groups;
    const uint64_t step = (uint64_t)gridDim.x * UNITS;
    uint64_t i = (uint64_t)blockIdx.x * UNITS + threadIdx.x / LANES;
    uint32_t token = i < n ? token_of(a, i) : 0;
    int32_t slot = i < n ? __ldg(a.slots + token) : -1;
    for (; i < n; i += step) {
        const Unit u = unit_of<H>(a, i, token, slot, lane);
        uint4 v[H][2];
#pragma unroll
        for (uint32_t h = 0; h < H; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                v[h][j] = make_uint4(0, 0, 0, 0);
                if (u.live && h < u.n) v[h][j] = ld_stream16(u.rows + h * (Q8_D / 8) + j * LANES);
            }
        if (i + step < n) {
            token = token_of(a, i + step);
            slot = __ldg(a.slots + token);
        }
        if (!u.live) continue;  // padding (the unit's lanes as one)
#pragma unroll
        for (uint32_t h = 0; h < H; ++h) {
            if (h >= u.n) break;
            uint32_t w[8] = {v[h][0].x, v[h][0].y, v[h][0].z, v[h][0].w, v[h][1].x, v[h][1].y, v[h][1].z, v[h][1].w};
            uint32_t mx = w[0] & 0x7fff7fffu;
#pragma unroll
            for (int j = 1; j < 8; ++j) mx = max_nan_bf16x2(mx, w[j] & 0x7fff7fffu);
#pragma unroll
            for (int o = LANES / 2; o >= 1; o >>= 1) mx = max_nan_bf16x2(mx, __shfl_xor_sync(group, mx, o));
            // Magnitudes order as their bits (a NaN above all).
            const uint32_t amax = max(mx & 0xffffu, mx >> 16);
            const bool finite = amax < 0x7f80u;
            if (amax > kQ8Top<FMT>) {  // rare
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = q8_below_2_128<FMT>(w[j]);
            }
            const int e = q8_exponent<FMT>(amax);
            const float inv = __uint_as_float((uint32_t)(127 - (finite ? e : 0)) << 23);
            uint8_t *codes = u.codes + (int64_t)h * a.block * Q8_D;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint2 c;
                c.x = q8_encode4<FMT>(w[4 * j], w[4 * j + 1], inv);
                c.y = q8_encode4<FMT>(w[4 * j + 2], w[4 * j + 3], inv);
                if (!finite) c = make_uint2(0, 0);
                *reinterpret_cast<uint2 *>(codes + j * (Q8_D / 2)) = c;
            }
            if (lane == 0) u.scale[(int64_t)h * a.block] = (uint8_t)(finite ? e + 127 : 255);
        }
    }
}

template <int FMT, uint32_t H>
__global__ void __launch_bounds__(Q8_THREADS) load_kvcache_q8_kernel(const Q8Rows a) {
    pdl_wait_then_release();
    const int lane = threadIdx.x % LANES;
    const uint64_t n = 2ull * a.num_tokens * a.groups;
    const uint64_t step = (uint64_t)gridDim.x * UNITS;
    uint64_t i = (uint64_t)blockIdx.x * UNITS + threadIdx.x / LANES;
    uint32_t token = i < n ? token_of(a, i) : 0;
    int32_t slot = i < n ? __ldg(a.slots + token) : -1;
    for (; i < n; i += step) {
        const Unit u = unit_of<H>(a, i, token, slot, lane);
        uint2 c[H][2];
        uint32_t s[H];
#pragma unroll
        for (uint32_t h = 0; h < H; ++h) {
            c[h][0] = c[h][1] = make_uint2(0, 0);  // a negative (or bad) slot reads as zeros
            s[h] = 127;
            if (u.live && h < u.n) {
                const uint2 *codes = reinterpret_cast<const uint2 *>(u.codes + (int64_t)h * a.block * Q8_D);
                c[h][0] = __ldg(codes);
                c[h][1] = __ldg(codes + LANES);
                s[h] = __ldg(u.scale + (int64_t)h * a.block);
            }
        }
        if (i + step < n) {
            token = token_of(a, i + step);
            slot = __ldg(a.slots + token);
        }
#pragma unroll
        for (uint32_t h = 0; h < H; ++h) {
            if (h >= u.n) break;
            const uint32_t sc = q8_scale_bf16x2(s[h]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint2 x = q8_to_bf16<FMT>(c[h][j].x, sc), y = q8_to_bf16<FMT>(c[h][j].y, sc);
                u.rows[h * (Q8_D / 8) + j * LANES] = make_uint4(x.x, x.y, y.x, y.y);
            }
        }
    }
}

// Units of H rows where a token has that many and each SM gets a CTA of them;
// smaller calls take units of one row, which more SMs share.  With 8 heads, units
// of one row or of H: 64 tokens stored in 1.8 or 2.2 us, 1000 in 3.0 or 2.5,
// 16384 in 20.9 or 19.0; 100 loaded in 1.8 or 2.3 (four), 1000 in 2.6 or 2.3 (two),
// 2000 in 3.5, 3.6 (two) or 3.1, 16384 in 17.0, 15.8 or 14.9.  Fewer heads, 65536
// tokens loaded: one head in 8.9 or 11.6 (four), two in 17.3, 15.9 or 17.3.
template <uint32_t H>
bool units_of(const Q8Rows &a, int sms) {
    return a.hkv >= H && 2LL * a.num_tokens * ((a.hkv + H - 1) / H) >= (int64_t)UNITS * sms;
}
// Eight lanes per unit and step, at most `most` CTAs per SM.  A long load, whose
// time is in its writes, gains from many short CTAs (262144 tokens: 265 us with
// 8, 245 with 16, 239 with 32, 237 with 64); a store of 65536 tokens takes 80 us
// with 8, 71 with 16 and 70 with 64, one of 16384 20.6, 19.1 and 19.6.
template <uint32_t H>
dim3 rows_grid(Q8Rows &a, int64_t most, int sms) {
    a.groups = (a.hkv + H - 1) / H;
    const int64_t units = 2LL * a.num_tokens * a.groups;
    return dim3((unsigned)std::min<int64_t>((units + UNITS - 1) / UNITS, most * sms));
}
template <int FMT, uint32_t H>
pa_status launch_store(Q8Rows a, int sms, cudaStream_t stream) {
    const dim3 grid = rows_grid<H>(a, 16, sms);
    return launch_pdl(store_kvcache_q8_kernel<FMT, H>, grid, dim3(Q8_THREADS), 0, stream, "store_kvcache_q8_kernel", a);
}
template <int FMT, uint32_t H>
pa_status launch_load(Q8Rows a, int sms, cudaStream_t stream) {
    const dim3 grid = rows_grid<H>(a, 64, sms);
    return launch_pdl(load_kvcache_q8_kernel<FMT, H>, grid, dim3(Q8_THREADS), 0, stream, "load_kvcache_q8_kernel", a);
}

template <int FMT>
pa_status launch_rows(const Q8Rows &a, bool store, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    if (store) return units_of<2>(a, sms) ? launch_store<FMT, 2>(a, sms, stream) : launch_store<FMT, 1>(a, sms, stream);
    if (units_of<4>(a, sms)) return launch_load<FMT, 4>(a, sms, stream);
    return units_of<2>(a, sms) ? launch_load<FMT, 2>(a, sms, stream) : launch_load<FMT, 1>(a, sms, stream);
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
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return format == PA_Q8_E4M3 ? launch_rows<PA_Q8_E4M3>(a, store, s) : launch_rows<PA_Q8_INT8>(a, store, s);
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
