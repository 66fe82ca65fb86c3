// pa_decode_q8.cu -- paged GQA decode attention over an 8-bit KV pool.
//
// What it computes: for sequence b, query head h (kv head g = h / G),
//   out[b,h] = softmax_p(scale * q[b,h].K[p]) V[p],
//   K[p] = kc[p] * 2^(ks[p]-127),  V[p] = vc[p] * 2^(vs[p]-127),  p < ctx_b.
//
// How (GB300 design):
//  * The work is a flat list of 32-key tiles ordered (sequence, kv head, tile).
//    It is cut into equal contiguous ranges, one per WARP of a persistent grid
//    (one CTA per SM).  A warp is its own producer: its lane 0 issues the TMA
//    copies of its next tiles into the warp's own ring of shared memory (K and
//    V codes, 4 KB each, 128-byte swizzled, and the 32 + 32 scale bytes) and
//    the warp waits on its own mbarriers.  No barrier between warps while it
//    streams: with half the bytes per key of a bf16 pool, the merges and
//    hand-overs of a CTA-wide pipeline would weigh twice as much.
//  * Q.K and P.V run as mma.sync m16n8k16 (fp16 in, fp32 accumulate) with the
//    KEYS (Q.K) and the VALUE DIMS (P.V) as the M side and the G <= 8 query
//    heads as N = 8: half the MMAs of the layout with heads as M.  The codes
//    are widened to fp16 in registers, exactly (hardware conversion of E4M3,
//    permute and packed subtract for INT8).  One ldmatrix register holds four
//    dims of a key, or two dims of two keys (.trans); the order in which the
//    MMA wants them is met by permuting the dims of q and of the output.
//  * q is brought to fp16 by a power of two per head (exact but for elements
//    below 2^-14 of the head's largest, off by at most 2^-25 of that).
//  * V's scale is folded into the exponent of its weight:
//    P'_p = 2^(x_p + vs_p - 127 - mv) with a running reference mv of its own,
//    so the fp16 weights are relative to the largest weighted row, which is
//    kept between 2^7 and 2^15 (a weight 2^-21 below it is still a normal
//    fp16 number, one 2^-32 below it rounds to 0); the softmax sum uses the
//    plain weights 2^(x_p - m) in fp32.
//  * Segment end: a pair (b, g) inside the warp's range is written directly; a
//    part goes to the workspace and the last arriving warp merges the pair's
//    parts in order, so the result does not depend on timing.
//  * All waits are bounded; a timeout records PA_DEV_TIMEOUT and ends the warp.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int KT = 32;            // keys per tile
constexpr int NW = 12;            // warps per CTA
constexpr int ST = 2;             // tiles in a warp's ring
constexpr int NT = NW * 32;
constexpr int TILE_BYTES = KT * Q8_D;                 // K or V codes of a tile
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int kMaxBatch = 2048;
constexpr int kMaxGrid = 160;     // CTAs of the persistent grid (min(SMs, this))
constexpr int kMaxWorkers = kMaxGrid * NW;
constexpr float kLazyRescale = 8.f;  // log2 headroom before a running reference must move
constexpr float kWeightTop = 7.f;    // log2 of the largest fp16 weight when its reference moves
constexpr unsigned FULL = 0xffffffffu;

constexpr int OFF_SC = NW * ST * STAGE_BYTES;         // scale bytes [NW][ST][2][KT]
constexpr int OFF_BAR = OFF_SC + NW * ST * 2 * KT;    // mbarriers [NW][ST]
constexpr int OFF_ZERO = OFF_BAR + NW * ST * 8;       // a row of zeros
constexpr int OFF_WSUM = OFF_ZERO + Q8_D;             // scan scratch [NW]
constexpr int OFF_CUM = OFF_WSUM + 64;                // tile prefix sum [batch + 1]
static_assert(OFF_SC % 16 == 0 && OFF_BAR % 8 == 0 && OFF_ZERO % 16 == 0 && NW * 4 <= 64, "shared-memory layout");
__host__ __device__ constexpr size_t off_ctx(int batch) { return OFF_CUM + 4 * (size_t)(batch + 1); }
constexpr size_t smem_bytes(int batch) { return off_ctx(batch) + 4 * (size_t)batch + 1024; }
static_assert(smem_bytes(kMaxBatch) <= 232448, "shared memory budget");

// Workspace: per worker two parts (its first and its last segment) of G heads:
// o [2 * kMaxWorkers][G][128] fp32, (m, mv, l, -) [2 * kMaxWorkers][G] float4,
// then the arrival counters [kMaxWorkers].
struct WsLayout {
    size_t ml_off, o_off, cnt_off, total;
};
WsLayout ws_layout(int G) {
    WsLayout w;
    w.o_off = 0;
    w.ml_off = (size_t)2 * kMaxWorkers * G * Q8_D * 4;
    w.cnt_off = w.ml_off + (size_t)2 * kMaxWorkers * G * 16;
    w.total = w.cnt_off + (size_t)kMaxWorkers * 4;
    return w;
}

struct Args {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    int64_t q_row_stride;
    const uint8_t *k_scale, *v_scale;
    const int32_t *block_tables;
    const int32_t *ctx_lens;
    int32_t max_blocks, batch, Hq, Hkv, block_size, box_rows, num_blocks;
    float scale_log2;
    int32_t ctx_limit;
    float *ws_o;
    float4 *ws_ml;
    int *ws_cnt;
    DevError *err;
    int32_t checked;
};

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// D += A.B, m16n8k16, fp16 in, fp32 accumulate.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// Transposes an 8x8 matrix of 16-bit elements held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
// The bytes (d0 k0, d1 k0, d0 k1, d1 k1) of a transposed V register as the two
// fp16 pairs (k0, k1) of dim d0 and of dim d1.
template <int FMT>
__device__ __forceinline__ void v_to_f16(uint32_t w, uint32_t &d0, uint32_t &d1) {
    q8_to_f16<FMT>(__byte_perm(w, 0, 0x3120), d0, d1);
}

// A position of the flat list.
struct Pos {
    int b, g, t, nt;
};

struct Shared {
    const uint32_t *cum;
    const int *ctx;
};

__device__ __forceinline__ Pos locate(const Args &a, const Shared &s, long long x) {
    const uint32_t qv = (uint32_t)(x / a.Hkv);
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.cum[mid] <= qv) lo = mid; else hi = mid - 1;
    }
    Pos p;
    p.b = lo;
    p.nt = (int)(s.cum[lo + 1] - s.cum[lo]);
    const long long off = x - (long long)a.Hkv * s.cum[lo];
    p.g = (int)(off / p.nt);
    p.t = (int)(off - (long long)p.g * p.nt);
    return p;
}

// The next tile's position (not past the list's end: the caller counts).
__device__ __forceinline__ void advance(const Args &a, const Shared &s, Pos &p) {
    if (++p.t < p.nt) return;
    p.t = 0;
    if (++p.g < a.Hkv) return;
    p.g = 0;
    do ++p.b; while (p.b < a.batch && s.ctx[p.b] == 0);
    if (p.b < a.batch) p.nt = (s.ctx[p.b] + KT - 1) / KT;
}

template <int G, int FMT>
__global__ void __launch_bounds__(NT, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint32_t *cum = reinterpret_cast<uint32_t *>(smem + OFF_CUM);
    int *ctx_s = reinterpret_cast<int *>(smem + off_ctx(a.batch));
    uint32_t *wsum = reinterpret_cast<uint32_t *>(smem + OFF_WSUM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + OFF_BAR) + warp * ST;
    uint8_t *ring = smem + warp * ST * STAGE_BYTES;
    uint8_t *ring_sc = smem + OFF_SC + warp * ST * 2 * KT;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NW * ST; ++i) mbar_init(reinterpret_cast<uint64_t *>(smem + OFF_BAR) + i, 1);
        fence_mbar_init();
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    if (threadIdx.x < Q8_D / 16) *reinterpret_cast<uint4 *>(smem + OFF_ZERO + 16 * threadIdx.x) = make_uint4(0, 0, 0, 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Context lengths and the exclusive prefix sum of the tile counts (per kv head).
    {
        const int per = (a.batch + NT - 1) / NT;
        const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
        uint32_t run = 0;
        for (int b = b0; b < b1; ++b) {
            int ctx = __ldg(a.ctx_lens + b);
            if (ctx < 0 || ctx > a.ctx_limit) {
                if (blockIdx.x == 0) record_error(a.err, PA_DEV_BAD_CONTEXT, b);
                ctx = ctx < 0 ? 0 : a.ctx_limit;
            }
            ctx_s[b] = ctx;
            run += (uint32_t)((ctx + KT - 1) / KT);
        }
        uint32_t x = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(FULL, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        uint32_t excl = x - run;
        for (int w = 0; w < warp; ++w) excl += wsum[w];
        for (int b = b0; b < b1; ++b) {
            cum[b] = excl;
            excl += (uint32_t)((ctx_s[b] + KT - 1) / KT);
        }
        if (threadIdx.x == NT - 1) cum[a.batch] = excl;
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Shared sh{cum, ctx_s};

    // Sequences with no context produce zeros.
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        if (ctx_s[b] != 0) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + (int64_t)b * a.Hq * Q8_D);
        for (int j = threadIdx.x; j < a.Hq * Q8_D / 8; j += NT) o[j] = make_uint4(0, 0, 0, 0);
    }

    // This worker's range.  Workers are numbered across the CTAs first, so a
    // short list spreads over the SMs.
    const long long total = (long long)a.Hkv * cum[a.batch];
    const int workers = (int)gridDim.x * NW, me = warp * (int)gridDim.x + (int)blockIdx.x;
    const long long base = total / workers, rem = total % workers;
    auto start_of = [&](int w) -> long long { return (long long)w * base + min((long long)w, rem); };
    auto owner_of = [&](long long x) -> int {
        const long long cut = rem * (base + 1);
        return (int)(x < cut ? x / (base + 1) : rem + (x - cut) / base);
    };
    const long long x_begin = start_of(me), x_end = start_of(me + 1);
    if (x_begin >= x_end) return;

    // ---- producer side: the tile at `ip` is issued next, its block ids are in
    // `blk` (lane 0: the first box, lane 1: the second when boxes have 16 rows).
    const uint64_t pol = policy_evict_first();
    Pos ip = locate(a, sh, x_begin);
    long long ix = x_begin;
    const int nbox = KT / a.box_rows;
    auto fetch = [&](const Pos &p) -> int {
        const int key = p.t * KT + (lane < nbox ? lane : 0) * a.box_rows;
        return key < ctx_s[p.b] ? __ldg(a.block_tables + (int64_t)p.b * a.max_blocks + key / a.block_size) : -1;
    };
    int blk = fetch(ip);
    auto issue = [&](int stage) {
        const int live = ctx_s[ip.b] - ip.t * KT;  // keys of the tile
        const int n = min(nbox, (live + a.box_rows - 1) / a.box_rows);
        const int blk1 = __shfl_sync(FULL, blk, 1);
        if (lane == 0) {
            uint8_t *st = ring + stage * STAGE_BYTES, *sc = ring_sc + stage * 2 * KT;
            uint32_t bytes = 0;
            for (int i = 0; i < n; ++i) {
                const int id = i ? blk1 : blk;
                bytes += 2 * a.box_rows * Q8_D + (id >= 0 && id < a.num_blocks ? 2 * a.box_rows : 0);
            }
            // Expected before any copy is issued.
            mbar_arrive_expect_tx(&bar[stage], bytes);
            for (int i = 0; i < n; ++i) {
                const int id = i ? blk1 : blk, key = ip.t * KT + i * a.box_rows;
                const bool good = id >= 0 && id < a.num_blocks;
                if (!good && a.checked)
                    record_error(a.err, PA_DEV_BAD_BLOCK, (long long)ip.b * a.max_blocks + key / a.block_size);
                // An invalid block reads as zeros: TMA fills rows out of range.
                const int64_t row = good ? ((int64_t)id * a.Hkv + ip.g) * a.block_size + key % a.block_size
                                         : -2LL * a.box_rows;
                uint8_t *kd = st + i * a.box_rows * Q8_D;
                tma_load_2d(kd, &tmk, 0, (int)row, &bar[stage], pol);
                tma_load_2d(kd + TILE_BYTES, &tmv, 0, (int)row, &bar[stage], pol);
                if (good) {
                    bulk_load(sc + i * a.box_rows, a.k_scale + row, (uint32_t)a.box_rows, &bar[stage]);
                    bulk_load(sc + KT + i * a.box_rows, a.v_scale + row, (uint32_t)a.box_rows, &bar[stage]);
                } else {
                    for (int j = 0; j < a.box_rows; j += 16) {
                        *reinterpret_cast<uint4 *>(sc + i * a.box_rows + j) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(sc + KT + i * a.box_rows + j) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();  // a later copy overwrites these bytes
                }
            }
        }
        __syncwarp();
        if (++ix < x_end) {
            advance(a, sh, ip);
            blk = fetch(ip);
        }
    };
    int issued = 0;
    for (; issued < ST && ix < x_end; ++issued) issue(issued);

    // ---- consumer side.  Fragment coordinates (m16n8k16): g4 = lane / 4 is a
    // key (Q.K) or a dim (P.V) row, t4 = lane % 4; columns 2*t4, 2*t4+1 are the
    // heads of the accumulators, column g4 the head of a B fragment.
    const int g4 = lane >> 2, t4 = lane & 3, r8 = lane & 7, mi = lane >> 3;
    const uint32_t zero_row = smem_addr(smem + OFF_ZERO);
    const bool h0 = 2 * t4 < G, h1 = 2 * t4 + 1 < G;  // this lane's two heads exist
    Pos p = locate(a, sh, x_begin);
    long long x = x_begin;
    int n = 0;  // tiles consumed
    while (x < x_end) {
        const int take = (int)min((long long)(p.nt - p.t), x_end - x);
        const int ctx = ctx_s[p.b];
        const int64_t bh0 = (int64_t)p.b * a.Hq + (int64_t)p.g * G;
        // q: chunk c's registers hold dims 16c + 4*t4 .. +3 of head g4.
        uint32_t qb[8][2];
        float qs0, qs1;
        {
            uint2 w[8];
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                w[c] = make_uint2(0, 0);
                if (g4 < G)
                    w[c] = __ldg(reinterpret_cast<const uint2 *>(a.q + (int64_t)p.b * a.q_row_stride +
                                                                 ((int64_t)p.g * G + g4) * Q8_D + 16 * c + 4 * t4));
                // Finite magnitudes order as their bits, NaN and infinity above.
                mx = max(max(mx, w[c].x & 0x7fffu), max((w[c].x >> 16) & 0x7fffu, max(w[c].y & 0x7fffu, (w[c].y >> 16) & 0x7fffu)));
            }
            mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
            mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
            // 2^-e brings the largest magnitude to [1, 2) ([2, 4) at the top of the range).
            const int e = min(max((int)(mx >> 7), 1), 253) - 127;
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                qb[c][0] = pack_f16(bf16lo(w[c].x) * f, bf16hi(w[c].x) * f);
                qb[c][1] = pack_f16(bf16lo(w[c].y) * f, bf16hi(w[c].y) * f);
            }
            // The factor of heads 2*t4, 2*t4+1 (head h is held by lanes 4h..4h+3).
            const float s = __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
            qs0 = __shfl_sync(FULL, s, 8 * t4);
            qs1 = __shfl_sync(FULL, s, 8 * t4 + 4);
        }
        float o[8][4];
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, mv0 = -INFINITY, mv1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        for (int i = 0; i < take; ++i, ++n) {
            const int stage = n % ST;
            if (!mbar_wait(&bar[stage], (n / ST) & 1)) {
                if (lane == 0) record_error(a.err, PA_DEV_TIMEOUT, 500 + warp);
                // Let the copies already issued land before shared memory goes away.
                for (int j = n + 1; j < issued; ++j) (void)mbar_wait(&bar[j % ST], (j / ST) & 1);
                return;
            }
            const uint32_t ks = smem_addr(ring + stage * STAGE_BYTES), vs = ks + TILE_BYTES;
            const uint32_t scs = smem_addr(ring_sc + stage * 2 * KT);
            const int nvalid = min(KT, ctx - (p.t + i) * KT);
#pragma unroll
            for (int grp = 0; grp < KT / 16; ++grp) {
                if (grp * 16 >= nvalid) break;
                // ---- S^T = K.Q^T for 16 keys
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t krow = ks + (uint32_t)(grp * 16 + (mi & 1) * 8 + r8) * Q8_D;
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    uint32_t r[4], a0, a1, a2, a3;
                    ldsm_x4(krow + (uint32_t)(((c + (mi >> 1)) ^ r8) << 4), r);
                    q8_to_f16<FMT>(r[0], a0, a2);
                    q8_to_f16<FMT>(r[1], a1, a3);
                    mma16816(s, a0, a1, a2, a3, qb[c][0], qb[c][1]);
                    q8_to_f16<FMT>(r[2], a0, a2);
                    q8_to_f16<FMT>(r[3], a1, a3);
                    mma16816(s, a0, a1, a2, a3, qb[c + 1][0], qb[c + 1][1]);
                }
                // ---- scores and weights of keys key0 (s[0], s[1]) and key0 + 8
                const int key0 = grp * 16 + g4, key1 = key0 + 8;
                const float k0 = q8_scale(ld_shared_u8(scs + key0)), k1 = q8_scale(ld_shared_u8(scs + key1));
                const uint32_t e0 = ld_shared_u8(scs + KT + key0), e1 = ld_shared_u8(scs + KT + key1);
                const float v0 = e0 == 255 ? NAN : (float)((int)e0 - 127), v1 = e1 == 255 ? NAN : (float)((int)e1 - 127);
                const bool ok0 = key0 < nvalid, ok1 = key1 < nvalid;
                float xx[4], yy[4];
                xx[0] = ok0 ? s[0] * k0 * qs0 : -INFINITY;
                xx[1] = ok0 ? s[1] * k0 * qs1 : -INFINITY;
                xx[2] = ok1 ? s[2] * k1 * qs0 : -INFINITY;
                xx[3] = ok1 ? s[3] * k1 * qs1 : -INFINITY;
                yy[0] = ok0 ? xx[0] + v0 : -INFINITY;
                yy[1] = ok0 ? xx[1] + v0 : -INFINITY;
                yy[2] = ok1 ? xx[2] + v1 : -INFINITY;
                yy[3] = ok1 ? xx[3] + v1 : -INFINITY;
                float tx0 = fmaxf(xx[0], xx[2]), tx1 = fmaxf(xx[1], xx[3]);
                float ty0 = fmaxf(yy[0], yy[2]), ty1 = fmaxf(yy[1], yy[3]);
                const bool move = (h0 && (tx0 > m0 + kLazyRescale || ty0 > mv0 + (kWeightTop + kLazyRescale))) ||
                                  (h1 && (tx1 > m1 + kLazyRescale || ty1 > mv1 + (kWeightTop + kLazyRescale)));
                if (__any_sync(FULL, move)) {
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1) {
                        tx0 = fmaxf(tx0, __shfl_xor_sync(FULL, tx0, d));
                        tx1 = fmaxf(tx1, __shfl_xor_sync(FULL, tx1, d));
                        ty0 = fmaxf(ty0, __shfl_xor_sync(FULL, ty0, d));
                        ty1 = fmaxf(ty1, __shfl_xor_sync(FULL, ty1, d));
                    }
                    auto moved = [](float &ref, float seen) -> float {  // 2^(old - new)
                        const float nw = fmaxf(ref, seen), f = nw == -INFINITY ? 1.f : fast_exp2(ref - nw);
                        ref = nw;
                        return f;
                    };
                    l0 *= moved(m0, tx0);
                    l1 *= moved(m1, tx1);
                    const float f0 = moved(mv0, ty0 - kWeightTop), f1 = moved(mv1, ty1 - kWeightTop);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        o[c][0] *= f0;
                        o[c][1] *= f1;
                        o[c][2] *= f0;
                        o[c][3] *= f1;
                    }
                }
                // A head with nothing finite yet keeps the reference 0 (its weights are 0 or NaN).
                const float um0 = m0 == -INFINITY ? 0.f : m0, um1 = m1 == -INFINITY ? 0.f : m1;
                const float uv0 = mv0 == -INFINITY ? 0.f : mv0, uv1 = mv1 == -INFINITY ? 0.f : mv1;
                l0 += fast_exp2(xx[0] - um0) + fast_exp2(xx[2] - um0);
                l1 += fast_exp2(xx[1] - um1) + fast_exp2(xx[3] - um1);
                // ---- O^T += V^T.P'^T; the weights become the B fragment by a transpose
                const uint32_t b0 = transpose8x8(pack_f16(fast_exp2(yy[0] - uv0), fast_exp2(yy[1] - uv1)));
                const uint32_t b1 = transpose8x8(pack_f16(fast_exp2(yy[2] - uv0), fast_exp2(yy[3] - uv1)));
                // Rows past the context may hold anything (NaN codes included) and
                // 0 * NaN is not 0: their lanes read the row of zeros.
                const int vk = grp * 16 + (mi & 1) * 8 + r8;
                const uint32_t vrow = vk < nvalid ? vs + (uint32_t)vk * Q8_D : zero_row;
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    uint32_t r[4], a0, a1, a2, a3;
                    ldsm_x4_t(vrow + (uint32_t)(((c + (mi >> 1)) ^ r8) << 4), r);
                    v_to_f16<FMT>(r[0], a0, a1);
                    v_to_f16<FMT>(r[1], a2, a3);
                    mma16816(o[c], a0, a1, a2, a3, b0, b1);
                    v_to_f16<FMT>(r[2], a0, a1);
                    v_to_f16<FMT>(r[3], a2, a3);
                    mma16816(o[c + 1], a0, a1, a2, a3, b0, b1);
                }
            }
            __syncwarp();  // every lane has read the stage
            if (ix < x_end) {
                issue(stage);
                ++issued;
            }
        }
        // ---- segment end.  This lane holds dims 16c + 2*g4, +1 of heads 2*t4, 2*t4+1.
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
            l0 += __shfl_xor_sync(FULL, l0, d);
            l1 += __shfl_xor_sync(FULL, l1, d);
        }
        if (p.t == 0 && take == p.nt) {
            const float f0 = fast_exp2(mv0 - m0) / l0, f1 = fast_exp2(mv1 - m1) / l1;
            __nv_bfloat16 *dst = a.out + (bh0 + 2 * t4) * Q8_D + 2 * g4;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (h0) *reinterpret_cast<__nv_bfloat162 *>(dst + 16 * c) = __floats2bfloat162_rn(o[c][0] * f0, o[c][2] * f0);
                if (h1) *reinterpret_cast<__nv_bfloat162 *>(dst + Q8_D + 16 * c) = __floats2bfloat162_rn(o[c][1] * f1, o[c][3] * f1);
            }
        } else {
            // A part of the pair: only a range's first and last segments can be.
            const int slot = 2 * me + (x == x_begin ? 0 : 1);
            float *dst = a.ws_o + ((int64_t)slot * G + 2 * t4) * Q8_D + 2 * g4;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (h0) *reinterpret_cast<float2 *>(dst + 16 * c) = make_float2(o[c][0], o[c][2]);
                if (h1) *reinterpret_cast<float2 *>(dst + Q8_D + 16 * c) = make_float2(o[c][1], o[c][3]);
            }
            if (g4 == 0) {
                if (h0) a.ws_ml[(int64_t)slot * G + 2 * t4] = make_float4(m0, mv0, l0, 0.f);
                if (h1) a.ws_ml[(int64_t)slot * G + 2 * t4 + 1] = make_float4(m1, mv1, l1, 0.f);
            }
            const long long x0 = x - p.t;  // the pair's first tile
            const int w0 = owner_of(x0), w1 = owner_of(x0 + p.nt - 1);
            __threadfence();
            __syncwarp();
            int arrived = 0;
            if (lane == 0) arrived = atomicAdd(&a.ws_cnt[w0], 1);
            arrived = __shfl_sync(FULL, arrived, 0);
            if (arrived == w1 - w0) {  // the last part: merge them all, in order
                __threadfence();
                const int s0 = 2 * w0 + (x0 == start_of(w0) ? 0 : 1);
                for (int h = 0; h < G; ++h) {
                    float M = -INFINITY, MV = -INFINITY;
                    for (int w = w0 + lane; w <= w1; w += 32) {
                        const float4 ml = __ldcg(a.ws_ml + (int64_t)(w == w0 ? s0 : 2 * w) * G + h);
                        M = fmaxf(M, ml.x);
                        MV = fmaxf(MV, ml.y);
                    }
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        M = fmaxf(M, __shfl_xor_sync(FULL, M, d));
                        MV = fmaxf(MV, __shfl_xor_sync(FULL, MV, d));
                    }
                    float L = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int w = w0; w <= w1; ++w) {
                        const int64_t row = (int64_t)(w == w0 ? s0 : 2 * w) * G + h;
                        const float4 ml = __ldcg(a.ws_ml + row);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.ws_o + row * Q8_D) + lane);
                        const float fv = fast_exp2(ml.y - MV);
                        L = fmaf(ml.z, fast_exp2(ml.x - M), L);
                        acc.x = fmaf(v.x, fv, acc.x);
                        acc.y = fmaf(v.y, fv, acc.y);
                        acc.z = fmaf(v.z, fv, acc.z);
                        acc.w = fmaf(v.w, fv, acc.w);
                    }
                    const float f = fast_exp2(MV - M) / L;
                    __nv_bfloat162 *od = reinterpret_cast<__nv_bfloat162 *>(a.out + (bh0 + h) * Q8_D + 4 * lane);
                    od[0] = __floats2bfloat162_rn(acc.x * f, acc.y * f);
                    od[1] = __floats2bfloat162_rn(acc.z * f, acc.w * f);
                }
                if (lane == 0) a.ws_cnt[w0] = 0;  // ready for the next call
            }
        }
        x += take;
        if (x < x_end) {
            p.t += take - 1;
            advance(a, sh, p);
        }
    }
}

std::atomic<int> g_attr_done[64][8];

template <int G, int FMT>
pa_status launch(const Args &a, const CUtensorMap &tk, const CUtensorMap &tv, int grid, cudaStream_t st) {
    int dev = 0;
    cudaGetDevice(&dev);
    const int gi = (G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3) + 4 * FMT;
    if (dev >= 0 && dev < 64 && !g_attr_done[dev][gi].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(decode_q8_kernel<G, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)smem_bytes(kMaxBatch));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(decode_q8_kernel)");
        g_attr_done[dev][gi].store(1, std::memory_order_release);
    }
    return launch_pdl(decode_q8_kernel<G, FMT>, dim3((unsigned)grid), dim3(NT), smem_bytes(a.batch), st,
                      "decode_q8_kernel", tk, tv, a);
}

template <int FMT>
pa_status launch_g(int G, const Args &a, const CUtensorMap &tk, const CUtensorMap &tv, int grid, cudaStream_t st) {
    switch (G) {
        case 1: return launch<1, FMT>(a, tk, tv, grid, st);
        case 2: return launch<2, FMT>(a, tk, tv, grid, st);
        case 4: return launch<4, FMT>(a, tk, tv, grid, st);
        default: return launch<8, FMT>(a, tk, tv, grid, st);
    }
}

bool supported_group(int num_q_heads, int num_kv_heads) {
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads) return false;
    const int G = num_q_heads / num_kv_heads;
    return G == 1 || G == 2 || G == 4 || G == 8;
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_decode_q8_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
    if (head_dim != pa::Q8_D || !pa::supported_group(num_q_heads, num_kv_heads)) return 0;
    return pa::ws_layout(num_q_heads / num_kv_heads).total;
}

pa_status pa_decode_q8(void *out, const void *q, int64_t q_row_stride, const void *k_cache, const void *v_cache,
                       const void *k_scale, const void *v_scale, const int32_t *block_tables,
                       int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                       int32_t format, float softmax_scale, void *workspace, size_t workspace_bytes,
                       pa_stream_t stream) {
    using namespace pa;
    if (batch < 0) return fail(PA_ERR_INVALID_ARG, "batch < 0");
    if (batch == 0) return PA_OK;
    if (batch > kMaxBatch) return fail(PA_ERR_UNSUPPORTED, "batch %d > %d", batch, kMaxBatch);
    if (!out || !q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads)
        return fail(PA_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
    const int G = num_q_heads / num_kv_heads;
    if (!supported_group(num_q_heads, num_kv_heads))
        return fail(PA_ERR_UNSUPPORTED, "GQA group %d (supported: 1, 2, 4, 8)", G);
    pa_status st = q8_check_pool(format, num_kv_heads, head_dim, block_size, num_blocks);
    if (st != PA_OK) return st;
    if (max_blocks_per_seq <= 0) return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq must be positive");
    if ((int64_t)max_blocks_per_seq * block_size > 0x7fffffffLL - KT)
        return fail(PA_ERR_UNSUPPORTED, "table too large for 32-bit positions");
    // The per-head tile prefix sum is 32-bit: batch * ceil(max_blocks * B / 32) must fit.
    if ((int64_t)batch * (((int64_t)max_blocks_per_seq * block_size + KT - 1) / KT) >= 0x7fffffffLL)
        return fail(PA_ERR_UNSUPPORTED, "batch x block-table capacity too large (%d x %lld tokens)", batch,
                    (long long)max_blocks_per_seq * block_size);
    if (q_row_stride < (int64_t)num_q_heads * Q8_D || q_row_stride % 8)
        return fail(PA_ERR_INVALID_ARG, "q_row_stride must be >= num_q_heads*head_dim and a multiple of 8");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) ||
        !aligned16(v_scale))
        return fail(PA_ERR_INVALID_ARG, "out/q/cache/scale pointers must be 16-byte aligned");
    if (!(softmax_scale > 0.f) || !isfinite(softmax_scale))
        return fail(PA_ERR_INVALID_ARG, "softmax_scale must be positive and finite");
    const WsLayout W = ws_layout(G);
    if (!workspace || workspace_bytes < W.total)
        return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", W.total,
                    workspace ? workspace_bytes : (size_t)0);
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");

    const int box = block_size % 32 ? 16 : 32;  // a TMA box stays inside a block
    const int64_t rows = (int64_t)num_blocks * num_kv_heads * block_size;
    CUtensorMap tk, tv;
    st = encode_row_map_u8(&tk, k_cache, rows, box);
    if (st != PA_OK) return st;
    st = encode_row_map_u8(&tv, v_cache, rows, box);
    if (st != PA_OK) return st;

    Args A;
    A.out = static_cast<__nv_bfloat16 *>(out);
    A.q = static_cast<const __nv_bfloat16 *>(q);
    A.q_row_stride = q_row_stride;
    A.k_scale = static_cast<const uint8_t *>(k_scale);
    A.v_scale = static_cast<const uint8_t *>(v_scale);
    A.block_tables = block_tables;
    A.ctx_lens = context_lens;
    A.max_blocks = max_blocks_per_seq;
    A.batch = batch;
    A.Hq = num_q_heads;
    A.Hkv = num_kv_heads;
    A.block_size = block_size;
    A.box_rows = box;
    A.num_blocks = num_blocks;
    A.scale_log2 = softmax_scale * 1.4426950408889634f;
    A.ctx_limit = max_blocks_per_seq * block_size;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    A.ws_o = reinterpret_cast<float *>(ws + W.o_off);
    A.ws_ml = reinterpret_cast<float4 *>(ws + W.ml_off);
    A.ws_cnt = reinterpret_cast<int *>(ws + W.cnt_off);
    A.err = device_error_ptr();
    A.checked = checked_mode() ? 1 : 0;
    const int grid = std::min(sm_count(), kMaxGrid);
    if (grid <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return format == PA_Q8_E4M3 ? launch_g<PA_Q8_E4M3>(G, A, tk, tv, grid, s)
                                : launch_g<PA_Q8_INT8>(G, A, tk, tv, grid, s);
}

}  // extern "C"
