// pa_decode_q8.cu -- paged GQA decode attention over an 8-bit KV pool.
//
// What it computes: for sequence b, query head h (kv head g = h / G),
//   out[b,h] = softmax_p(scale * q[b,h].K[p]) V[p],
//   K[p] = kc[p] * 2^(ks[p]-127),  V[p] = vc[p] * 2^(vs[p]-127),  p < ctx_b.
//
// How (GB300 design):
//  * The work is a flat list of 32-key tiles ordered (sequence, kv head, tile),
//    cut into contiguous ranges of equal cost, one per CTA of a persistent grid
//    (one CTA per SM), and each CTA's range likewise between its WARPS.  A pair
//    costs half a tile on top of its tiles (measured: 0.7 us where a tile takes
//    a warp 1.5 us).  A warp is its own producer: its lane 0 issues the TMA copies of
//    its next tiles into the warp's own ring of shared memory (K and V codes,
//    4 KB each, 128-byte swizzled) and the warp waits on its own mbarriers;
//    the scale bytes, one per lane, are plain loads a ring ahead.  No barrier between warps while they stream:
//    with half the bytes per key of a bf16 pool, the merges and hand-overs of
//    a CTA-wide pipeline would weigh twice as much.  Eight warps with two tiles
//    each (128 KB in flight per SM) fill the bandwidth; twelve only lengthen
//    the memory's queues, whose service then differs more between warps (long
//    contexts, E4M3: 93 us instead of 85).  Chunks of the last eighth, taken
//    from a counter by the warps that are done, even out the ends to 5 us but
//    cost more in pieces and merges than that (95 us).
//  * Q.K and P.V run as mma.sync m16n8k16 (fp16 in, fp32 accumulate) with the
//    KEYS (Q.K) and the VALUE DIMS (P.V) as the M side and the G <= 8 query
//    heads as N = 8: half the MMAs of the layout with heads as M.  The codes
//    are widened to fp16 in registers, exactly (hardware conversion of E4M3,
//    permute and packed subtract for INT8).  One ldmatrix register holds four
//    dims of a key, or two dims of two keys (.trans); the order in which the
//    MMA wants them is met by permuting the dims of q and of the output.
//  * q is brought to fp16 by a power of two per head that takes its largest
//    element to the top of fp16's range: exact but for elements below 2^-31 of
//    that, which are off by at most 2^-39 of it (fp32 sums lose 2^-24).
//  * V's scale is folded into the exponent of its weight:
//    P'_p = 2^(x_p + vs_p - 127 - mv) with a running reference mv of its own,
//    so the fp16 weights are relative to the largest weighted row, which is
//    kept between 2^7 and 2^15 (a weight 2^-21 below it is still a normal
//    fp16 number, one 2^-32 below it rounds to 0); the softmax sum uses the
//    plain weights 2^(x_p - m) in fp32.
//  * A pair (b, g) inside a warp's range is written directly.  The pieces of
//    the others meet when the CTA's warps are done, one (pair, head) per warp
//    at a time; pairs that span CTAs leave a part in the workspace and the
//    CTA that arrives last merges them.  Pieces are combined in list order,
//    so the result does not depend on timing.  A pair is cut between at most
//    kMaxParts CTAs (or so), since its parts are read by one CTA.
//  * Fused store: the warp that has a pair's last tile loads the new token's K
//    and V row of that kv head when the segment begins, quantises them (four
//    values a lane), and puts codes and scale bytes into the landed tile and
//    into the pool.  Nothing else in the launch reads that slot.
//  * All waits are bounded; a timeout records PA_DEV_TIMEOUT and ends the warp.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int KT = 32;            // keys per tile
constexpr int NW = 8;             // warps per CTA
constexpr int ST = 2;             // tiles in a warp's ring
constexpr int NT = NW * 32;
constexpr int NG = KT / 16;       // MMA key groups of a tile
constexpr int TILE_BYTES = KT * Q8_D;                 // K or V codes of a tile
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int kMaxBatch = 2048;
constexpr int kMaxGrid = 160;     // CTAs of the persistent grid (min(SMs, this))
// CTAs that share a pair, about.  More stream a lone pair in less time and merge
// more parts at its end; 16, 32, 64 or 152 of them: one sequence of 32768 keys
// under one kv head 17.5, 13.7, 14.1 or 20.8 us, of 4096 keys 8.8, 9.5, 11.9 or
// 11.8, one of 32768 among 255 short ones (one kv head) 24.0, 18.5, 18.4 or 16.6,
// under eight kv heads 35.5 to 35.7; full batches and long contexts do not differ.
constexpr uint32_t kMaxParts = 32;
// Tiles of a CTA, at least (its range then holds the beginning of one): with 2, 4
// or 8, four sequences of 600 keys at most 7.6, 7.6 or 7.9 us, eight of 300 9.5,
// 9.5 or 10.1, four of 100 5.4, 5.3 or 5.9.
constexpr uint32_t kMinTilesPerCta = 2;
constexpr float kLazyRescale = 8.f;  // log2 headroom before a running reference must move
constexpr float kWeightTop = 7.f;    // log2 of the largest fp16 weight when its reference moves
constexpr unsigned FULL = 0xffffffffu;

constexpr int OFF_BAR = NW * ST * STAGE_BYTES;        // mbarriers [NW][ST]
constexpr int OFF_ZERO = OFF_BAR + NW * ST * 8;       // a row of zeros
constexpr int OFF_WSUM = OFF_ZERO + Q8_D;             // scan scratch [3][NW]
constexpr int OFF_PIECE = OFF_WSUM + 128;             // (b, g) of each warp's two pieces [2 * NW] (-1: none)
constexpr int OFF_ABORT = OFF_PIECE + 256;            // a wait ran out
constexpr int OFF_SPAN = OFF_ABORT + 16;              // the pairs that span CTAs: {first CTA, CTAs} [2]
constexpr int OFF_CUM = OFF_SPAN + 32;                // tile prefix sum [batch + 1]
static_assert(OFF_BAR % 16 == 0 && OFF_ZERO % 16 == 0 && NW * 12 <= 128, "shared-memory layout");
static_assert(NW <= 16, "a warp's lanes hold the CTA's pieces");
__host__ __device__ constexpr size_t off_cost(int batch) { return OFF_CUM + 4 * (size_t)(batch + 1); }  // cost prefix sum [batch + 1]
__host__ __device__ constexpr size_t off_ctx(int batch) { return off_cost(batch) + 4 * (size_t)(batch + 1); }
__host__ __device__ constexpr size_t off_stash(int batch) { return (off_ctx(batch) + 4 * (size_t)batch + 15) / 16 * 16; }

// A piece of a pair: o [G][128] fp32, then (m, mv, l, -) [G].  The pieces of the
// warps' ranges (first and last segment) are stashed in shared memory, a CTA's
// parts of pairs that span CTAs in the workspace.
template <int G>
constexpr int kPiece = G * (Q8_D + 4);  // floats
constexpr size_t smem_bytes(int batch, int G) {
    return off_stash(batch) + (size_t)2 * NW * G * (Q8_D + 4) * 4 + 1024;
}
constexpr size_t kMaxSmem = 232448;
static_assert(smem_bytes(kMaxBatch, 8) <= kMaxSmem, "shared memory budget");

// Workspace: the arrival counters [kMaxGrid][8] (of the heads of the pair that
// begins in a CTA's range and ends in a later one), then the CTAs' parts
// [kMaxGrid][2] (of the pair that began in an earlier range, of the one that
// begins in this range).  The counters, which a call finds and leaves zeroed,
// come first: their place does not depend on the group, so that calls of other
// groups, whose parts end elsewhere, never write over them.
constexpr size_t kWsParts = (size_t)kMaxGrid * 8 * 4;  // bytes before the parts
static_assert(kWsParts % 256 == 0, "the parts are read 16 bytes at a time");
size_t ws_bytes(int G) { return kWsParts + (size_t)2 * kMaxGrid * G * (Q8_D + 4) * 4; }

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
    // Fused store: the new token's rows (null: none) and the pool they go to.
    const uint2 *new_k, *new_v;
    int64_t new_k_stride, new_v_stride;  // in 8-byte units
    uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
    float *ws_part;
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
// The bytes (d0 k0, d1 k0, d0 k1, d1 k1) of a transposed V register as the two
// fp16 pairs (k0, k1) of dim d0 and of dim d1.
template <int FMT>
__device__ __forceinline__ void v_to_f16(uint32_t w, uint32_t &d0, uint32_t &d1) {
    if (FMT == PA_Q8_INT8) q8_int8_to_f16<0x4240, 0x4341>(w, d0, d1);
    else q8_to_f16<FMT>(__byte_perm(w, 0, 0x3120), d0, d1);
}

// Quantises the row whose values 4*lane .. +3 the warp's lanes hold (bf16): the
// lane's four codes, and the row's scale byte.
template <int FMT>
__device__ __forceinline__ uint32_t quantise_row(uint2 w, uint32_t &scale) {
    // Magnitudes order as their bits, infinities and NaN above all.
    uint32_t mx = max(max(w.x & 0x7fffu, (w.x >> 16) & 0x7fffu), max(w.y & 0x7fffu, (w.y >> 16) & 0x7fffu));
    mx = __reduce_max_sync(FULL, mx);
    if (mx >= 0x7f80u) {
        scale = 255;
        return 0;
    }
    if (mx > kQ8Top<FMT>) w = make_uint2(q8_below_2_128<FMT>(w.x), q8_below_2_128<FMT>(w.y));
    const int e = q8_exponent<FMT>(mx);
    scale = (uint32_t)(e + 127);
    return q8_encode4<FMT>(w.x, w.y, __uint_as_float((uint32_t)(127 - e) << 23));
}

// Adds to a counter: releases what the warp wrote before (ordered by its
// barrier), acquires what the earlier adders released.
__device__ __forceinline__ int add_acq_rel(int *p, int v) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// A position of the flat list.
struct Pos {
    int b, g, t, nt;
};

// Per sequence, in shared memory: prefix sums (per kv head) of the tiles and of
// the costs, and the context lengths.  Cost unit: half a tile; pair (b, g) has
// 2 * nt + 1 units, of which the first is its own and tile t begins at 1 + 2t.
struct Shared {
    const uint32_t *cum, *cost;
    const int *ctx;
};

// The first tile that begins at unit x or later: its position (b = batch past
// the end) and its index in the list.
__device__ __forceinline__ Pos locate(const Args &a, const Shared &s, uint32_t x, uint32_t &tile) {
    Pos p = {a.batch, 0, 0, 0};
    tile = (uint32_t)a.Hkv * s.cum[a.batch];
    if (x >= (uint32_t)a.Hkv * s.cost[a.batch]) return p;
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((uint32_t)a.Hkv * s.cost[mid] <= x) lo = mid; else hi = mid - 1;
    }
    p.b = lo;
    p.nt = (int)(s.cum[lo + 1] - s.cum[lo]);
    const uint32_t off = x - (uint32_t)a.Hkv * s.cost[lo], units = 2 * p.nt + 1;
    p.g = (int)(off / units);
    p.t = (int)(off - (uint32_t)p.g * units) / 2;
    tile = (uint32_t)a.Hkv * s.cum[lo] + (uint32_t)(p.g * p.nt + p.t);
    if (p.t == p.nt) {  // the pair's last tile begins before x
        p.t = 0;
        if (++p.g == a.Hkv) {
            p.g = 0;
            do ++p.b; while (p.b < a.batch && s.ctx[p.b] == 0);
            p.nt = p.b < a.batch ? (s.ctx[p.b] + KT - 1) / KT : 0;
        }
    }
    return p;
}

// The unit at which tile t of a pair begins.
__device__ __forceinline__ uint32_t unit_of(const Args &a, const Shared &s, const Pos &p, uint32_t t) {
    return (uint32_t)a.Hkv * s.cost[p.b] + (uint32_t)p.g * (2 * p.nt + 1) + 1 + 2 * t;
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

// The largest of a warp's values (none NaN), by one integer reduction each way:
// floats order as their bits with the sign bit, or all bits, flipped.
__device__ __forceinline__ float warp_max(float x) {
    const uint32_t b = __float_as_uint(x);
    const uint32_t m = __reduce_max_sync(FULL, (b >> 31) ? ~b : b | 0x80000000u);
    return __uint_as_float((m >> 31) ? m & 0x7fffffffu : ~m);
}

// Merges pieces of one pair and head: bit i of `mask` stands for the piece at
// base + index(i) * kPiece.  Every lane returns dims 4*lane .. +3 and the totals.
// FAR: the pieces are CTAs' parts (read from L2); else in shared memory.
struct Merged {
    float m, mv, l;
    float4 o;
};
template <bool FAR>
__device__ __forceinline__ float4 ld_piece(const float *p) {
    const float4 *v = reinterpret_cast<const float4 *>(p);
    return FAR ? __ldcg(v) : *v;
}
template <int G, bool FAR, typename Index>
__device__ __forceinline__ Merged merge_pieces(const float *base, Index index, unsigned mask, int h) {
    const int lane = threadIdx.x & 31;
    float4 ml = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
    if (mask >> lane & 1) ml = ld_piece<FAR>(base + (int64_t)index(lane) * kPiece<G> + G * Q8_D + 4 * h);
    constexpr int PF = FAR ? 8 : 4;  // pieces whose loads are in flight
    const float *mine = base + h * Q8_D + 4 * lane;
    Merged r;
    r.o = make_float4(0.f, 0.f, 0.f, 0.f);
    float f = 0.f;
    bool first = true;
#pragma unroll 1
    while (mask) {
        float4 v[PF];
        int from[PF];
#pragma unroll
        for (int u = 0; u < PF; ++u) {
            from[u] = mask ? __ffs(mask) - 1 : 32;
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mask) v[u] = ld_piece<FAR>(mine + (int64_t)index(from[u]) * kPiece<G>);
            mask &= mask - 1;
        }
        if (first) {  // behind the first loads
            first = false;
            r.m = warp_max(ml.x);
            r.mv = warp_max(ml.y);
            // 2^(own - max): a piece without a finite score has l = 0 or NaN.
            r.l = ml.z * (ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - r.m));
            f = ml.y == -INFINITY ? 1.f : fast_exp2(ml.y - r.mv);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) r.l += __shfl_xor_sync(FULL, r.l, d);
        }
#pragma unroll
        for (int u = 0; u < PF; ++u) {
            const float w = __shfl_sync(FULL, f, from[u] & 31);
            if (from[u] == 32) continue;
            r.o.x = fmaf(v[u].x, w, r.o.x);
            r.o.y = fmaf(v[u].y, w, r.o.y);
            r.o.z = fmaf(v[u].z, w, r.o.z);
            r.o.w = fmaf(v[u].w, w, r.o.w);
        }
    }
    return r;
}

// The factor of a key's and of a head's scale, at most the largest fp32 number
// (NaN kept).  The two are multiplied first: either alone may take a product of
// codes out of fp32's range although the score is an ordinary number.  Without
// the limit a product of 0 would become NaN where both are huge.
__device__ __forceinline__ float score_scale(float k, float q) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(k * q), "f"(3.402823466e38f));
    return r;
}

// 2^(mv - m) / l, by which a pair's sum of weighted codes becomes its output, in
// two factors: value rows near either end of bf16's range have exponents beyond
// fp32's (mv - m down to -142 and up to 128).  The second is 1, 2^64 or 2^-64, so
// that the others lose nothing.
struct OutScale {
    float f, far;
    __device__ float operator()(float o) const { return o * f * far; }
};
__device__ __forceinline__ OutScale out_scale(float m, float mv, float l) {
    const float e = mv - m, shift = e < -64.f ? -64.f : e > 64.f ? 64.f : 0.f;
    return {fast_exp2(e - shift) / l, shift < 0.f ? 0x1p-64f : shift > 0.f ? 0x1p64f : 1.f};
}

__device__ __forceinline__ void write_out(const Args &a, const Merged &r, int64_t row) {
    const OutScale f = out_scale(r.m, r.mv, r.l);
    __nv_bfloat162 *od = reinterpret_cast<__nv_bfloat162 *>(a.out + row * Q8_D + 4 * (threadIdx.x & 31));
    od[0] = __floats2bfloat162_rn(f(r.o.x), f(r.o.y));
    od[1] = __floats2bfloat162_rn(f(r.o.z), f(r.o.w));
}

// Merges the parts of a pair that n CTAs from c0 on share (it begins in c0's
// range) for head h, output row `row`.
template <int G>
__device__ void merge_parts(const Args &a, int64_t row, int c0, int n, int h) {
    Merged r;
    for (int i = 0; i < n; i += 32) {
        const int left = n - i;
        const Merged q = merge_pieces<G, true>(
            a.ws_part, [&](int j) { return 2 * (c0 + i + j) + (i + j == 0 ? 1 : 0); },
            left >= 32 ? FULL : (1u << left) - 1, h);
        if (i == 0) {
            r = q;
            continue;
        }
        const float m = fmaxf(r.m, q.m), mv = fmaxf(r.mv, q.mv);
        const float fr = r.m == -INFINITY ? 1.f : fast_exp2(r.m - m), fq = q.m == -INFINITY ? 1.f : fast_exp2(q.m - m);
        const float gr = r.mv == -INFINITY ? 1.f : fast_exp2(r.mv - mv), gq = q.mv == -INFINITY ? 1.f : fast_exp2(q.mv - mv);
        r.l = r.l * fr + q.l * fq;
        r.o.x = r.o.x * gr + q.o.x * gq;
        r.o.y = r.o.y * gr + q.o.y * gq;
        r.o.z = r.o.z * gr + q.o.z * gq;
        r.o.w = r.o.w * gr + q.o.w * gq;
        r.m = m;
        r.mv = mv;
    }
    write_out(a, r, row);
}

// Equal contiguous shares of n items (the list's length is bounded on the host,
// so that units fit 32 bits).
struct Split {
    uint32_t base, rem;
    __device__ Split(uint32_t n, uint32_t parts) : base(n / parts), rem(n - n / parts * parts) {}
    __device__ uint32_t start(uint32_t i) const { return i * base + min(i, rem); }
    __device__ uint32_t owner(uint32_t x) const {
        const uint32_t cut = rem * (base + 1);
        return x < cut ? x / (base + 1) : rem + (x - cut) / base;
    }
};

template <int G, int FMT>
__global__ void __launch_bounds__(NT, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint32_t *cum = reinterpret_cast<uint32_t *>(smem + OFF_CUM);
    uint32_t *cost = reinterpret_cast<uint32_t *>(smem + off_cost(a.batch));
    int *ctx_s = reinterpret_cast<int *>(smem + off_ctx(a.batch));
    uint32_t *wsum = reinterpret_cast<uint32_t *>(smem + OFF_WSUM);
    int2 *piece_pair = reinterpret_cast<int2 *>(smem + OFF_PIECE);
    int *abort = reinterpret_cast<int *>(smem + OFF_ABORT);
    int2 *span = reinterpret_cast<int2 *>(smem + OFF_SPAN);
    float *stash = reinterpret_cast<float *>(smem + off_stash(a.batch));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + OFF_BAR) + warp * ST;
    uint8_t *ring = smem + warp * ST * STAGE_BYTES;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NW * ST; ++i) mbar_init(reinterpret_cast<uint64_t *>(smem + OFF_BAR) + i, 1);
        fence_mbar_init();
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        *abort = 0;
    }
    if (threadIdx.x < Q8_D / 16) *reinterpret_cast<uint4 *>(smem + OFF_ZERO + 16 * threadIdx.x) = make_uint4(0, 0, 0, 0);
    if (threadIdx.x < 2 * NW) piece_pair[threadIdx.x] = make_int2(-1, 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Context lengths, their maximum, and the exclusive prefix sum of the tile
    // counts (per kv head).
    {
        const int per = (a.batch + NT - 1) / NT;
        const int b0 = min(a.batch, (int)threadIdx.x * per), b1 = min(a.batch, b0 + per);
        uint32_t run = 0, live = 0, top = 0;  // tiles, sequences that have some, most tiles
        for (int b = b0; b < b1; ++b) {
            int ctx = __ldg(a.ctx_lens + b);
            if (ctx < 0 || ctx > a.ctx_limit) {
                if (blockIdx.x == 0) record_error(a.err, PA_DEV_BAD_CONTEXT, b);
                ctx = ctx < 0 ? 0 : a.ctx_limit;
            }
            ctx_s[b] = ctx;
            const uint32_t nt = (uint32_t)((ctx + KT - 1) / KT);
            run += nt;
            live += nt ? 1u : 0u;
            top = max(top, nt);
        }
        uint32_t x = run, z = live;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(FULL, x, o), w = __shfl_up_sync(FULL, z, o);
            if (lane >= o) {
                x += y;
                z += w;
            }
        }
        top = __reduce_max_sync(FULL, top);
        if (lane == 31) {
            wsum[warp] = x;
            wsum[NW + warp] = top;
            wsum[2 * NW + warp] = z;
        }
        __syncthreads();
        uint32_t excl = x - run, seqs = z - live;
        for (int w = 0; w < warp; ++w) {
            excl += wsum[w];
            seqs += wsum[2 * NW + w];
        }
        for (int b = b0; b < b1; ++b) {
            cum[b] = excl;
            cost[b] = 2 * excl + seqs;
            const uint32_t nt = (uint32_t)((ctx_s[b] + KT - 1) / KT);
            excl += nt;
            seqs += nt ? 1u : 0u;
        }
        if (threadIdx.x == NT - 1) {
            cum[a.batch] = excl;
            cost[a.batch] = 2 * excl + seqs;
        }
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Shared sh{cum, cost, ctx_s};

    // Sequences with no context produce zeros.
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
        if (ctx_s[b] != 0) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + (int64_t)b * a.Hq * Q8_D);
        for (int j = threadIdx.x; j < a.Hq * Q8_D / 8; j += NT) o[j] = make_uint4(0, 0, 0, 0);
    }

    // The CTAs that work, and this one's range; then this warp's.
    const uint32_t total = (uint32_t)a.Hkv * cum[a.batch];
    uint32_t nt_max = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) nt_max = max(nt_max, wsum[NW + w]);
    const uint32_t least = max(kMinTilesPerCta, (nt_max + kMaxParts - 1) / kMaxParts);
    const uint32_t ctas = total >= gridDim.x * (uint64_t)least ? gridDim.x : (total + least - 1) / least;
    const uint32_t cta = blockIdx.x;
    if (cta >= ctas) return;
    const Split by_cta((uint32_t)a.Hkv * cost[a.batch], ctas);
    const uint32_t cu = by_cta.start(cta), cu_end = by_cta.start(cta + 1);
    const Split by_warp(cu_end - cu, NW);
    // Lanes 0 and 1 find the warp's first tile and the one after its last, lanes
    // 2 and 3 the CTA's.  A range of three units or more holds a tile; a CTA's
    // has more, a warp's may not.
    Pos ip;
    uint32_t x_begin, x_end, c_begin, c_end;
    Pos edge;            // lanes 2 and 3: the first tile at or after the CTA's ends
    uint32_t edge_pair;  // and the first tile of its pair
    {
        const uint32_t u = lane == 0 ? cu + by_warp.start(warp) : lane == 1 ? cu + by_warp.start(warp + 1) : lane == 2 ? cu : cu_end;
        uint32_t tile;
        const Pos e = locate(a, sh, u, tile);
        x_begin = __shfl_sync(FULL, tile, 0);
        x_end = __shfl_sync(FULL, tile, 1);
        c_begin = __shfl_sync(FULL, tile, 2);
        c_end = __shfl_sync(FULL, tile, 3);
        ip.b = __shfl_sync(FULL, e.b, 0);
        ip.g = __shfl_sync(FULL, e.g, 0);
        ip.t = __shfl_sync(FULL, e.t, 0);
        ip.nt = __shfl_sync(FULL, e.nt, 0);
        edge = e;
        edge_pair = tile - (uint32_t)e.t;
    }

    // The pairs that span CTAs: the one the range begins inside of, and the one it
    // ends inside of, if that began in it.
    auto note_spans = [&]() {
        if (warp == 0 && (lane == 2 || lane == 3) && edge.t > 0 && (lane == 2 || edge_pair >= c_begin)) {
            const int c0 = (int)by_cta.owner(unit_of(a, sh, edge, 0));
            span[lane - 2] = make_int2(c0, (int)by_cta.owner(unit_of(a, sh, edge, (uint32_t)edge.nt - 1)) - c0 + 1);
        }
    };
    if (x_begin >= x_end) {
        note_spans();
    } else {
        // ---- producer side: the tile at `ip` is issued next.  Lane i stands for its
        // key i; `blk` is the block that holds it.
        const uint64_t pol = policy_evict_first();
        Pos p = ip;
        uint32_t ix = x_begin;
        const bool two = a.box_rows < KT;  // boxes of 16 keys: lane 16 issues the second
        const int sub16 = two ? lane & 16 : 0;
        // The logical block and the offset in it of this lane's box, kept up tile
        // by tile: divisions only here (a pair starts at block 0).
        int lb = (int)((uint32_t)(ip.t * KT + sub16) / (uint32_t)a.block_size);
        int off = ip.t * KT + sub16 - lb * a.block_size;
        auto fetch = [&]() -> int {
            return ip.t * KT + sub16 < ctx_s[ip.b] ? __ldg(a.block_tables + (int64_t)ip.b * a.max_blocks + lb) : -1;
        };
        int blk = fetch();
        // The scale bytes of the tile being consumed and of the one behind it
        // (tile n's are loaded when its copy is issued, ST tiles ahead).
        uint32_t k_byte[ST], v_byte[ST];
        auto issue = [&](int stage, uint32_t &kb, uint32_t &vb) {
            const int key = ip.t * KT + lane, ctx = ctx_s[ip.b];
            const bool good = blk >= 0 && blk < a.num_blocks;
            // An invalid block reads as zeros: TMA fills rows out of range.
            const int64_t row = good ? ((int64_t)blk * a.Hkv + ip.g) * a.block_size + off + (lane - sub16) : -2LL * KT;
            kb = vb = 127;
            if (good && key < ctx) {
                kb = __ldg(a.k_scale + row);
                vb = __ldg(a.v_scale + row);
            }
            uint8_t *kd = ring + stage * STAGE_BYTES + lane * Q8_D;
            if (lane == 0) {  // expected before any copy is issued
                const int boxes = two && key + 16 < ctx ? 2 : 1;
                mbar_arrive_expect_tx(&bar[stage], (uint32_t)(boxes * 2 * a.box_rows * Q8_D));
            }
            if (two) __syncwarp();
            if (lane == 0 || (two && lane == 16 && key < ctx)) {
                if (!good && a.checked)
                    record_error(a.err, PA_DEV_BAD_BLOCK, (long long)ip.b * a.max_blocks + lb);
                tma_load_2d(kd, &tmk, 0, (int)row, &bar[stage], pol);
                tma_load_2d(kd + TILE_BYTES, &tmv, 0, (int)row, &bar[stage], pol);
            }
            __syncwarp();
            if (++ix < x_end) {
                advance(a, sh, ip);
                off += KT;
                bool other = false;  // another block
                while (off >= a.block_size) {
                    off -= a.block_size;
                    ++lb;
                    other = true;
                }
                if (ip.t == 0) {  // another pair
                    lb = sub16 < a.block_size ? 0 : 1;
                    off = sub16 - lb * a.block_size;
                    other = true;
                }
                if (other) blk = fetch();
            }
        };
        int issued = 0;
#pragma unroll
        for (int i = 0; i < ST; ++i)
            if (ix < x_end) issue(issued++, k_byte[i], v_byte[i]);
        note_spans();  // while the first tiles travel

        // ---- consumer side.  Fragment coordinates (m16n8k16): g4 = lane / 4 is a
        // key (Q.K) or a dim (P.V) row, t4 = lane % 4; columns 2*t4, 2*t4+1 are the
        // heads of the accumulators, column g4 the head of a B fragment.
        const int g4 = lane >> 2, t4 = lane & 3, r8 = lane & 7, mi = lane >> 3;
        const uint32_t zero_row = smem_addr(smem + OFF_ZERO);
        const bool h0 = 2 * t4 < G, h1 = 2 * t4 + 1 < G;  // this lane's two heads exist
        uint2 qw[8];
        auto load_q = [&](const Pos &q) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                qw[c] = make_uint2(0, 0);
                if (g4 < G)
                    qw[c] = __ldg(reinterpret_cast<const uint2 *>(a.q + (int64_t)q.b * a.q_row_stride +
                                                                  ((int64_t)q.g * G + g4) * Q8_D + 16 * c + 4 * t4));
            }
        };
        load_q(p);
        uint32_t x = x_begin;
        int n = 0;  // tiles consumed
        bool ok = true;
        while (ok && x < x_end) {
            const int take = (int)min((uint32_t)(p.nt - p.t), x_end - x);
            const int ctx = ctx_s[p.b];
            // q: chunk c's registers hold dims 16c + 4*t4 .. +3 of head g4.
            uint32_t qb[8][2];
            float qs0, qs1;
            {
                uint32_t mx = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    // Finite magnitudes order as their bits, NaN and infinity above.
                    mx = max(max(mx, qw[c].x & 0x7fffu), max((qw[c].x >> 16) & 0x7fffu,
                             max(qw[c].y & 0x7fffu, (qw[c].y >> 16) & 0x7fffu)));
                mx = max(mx, __shfl_xor_sync(FULL, mx, 1));
                mx = max(mx, __shfl_xor_sync(FULL, mx, 2));
                // 2^-e brings the largest magnitude to [2^14, 2^15).  A head below 2^-95 goes less
                // far, to multiples of 2^-24 (bf16's are of 2^-133), which fp16 holds exactly.
                const int e = min(max((int)(mx >> 7), 32), 254) - 127 - 14;
                const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    qb[c][0] = pack_f16(bf16lo(qw[c].x) * f, bf16hi(qw[c].x) * f);
                    qb[c][1] = pack_f16(bf16lo(qw[c].y) * f, bf16hi(qw[c].y) * f);
                }
                // The factor of heads 2*t4, 2*t4+1 (head h is held by lanes 4h..4h+3).
                const float s = __uint_as_float((uint32_t)(127 + e) << 23) * a.scale_log2;
                qs0 = __shfl_sync(FULL, s, 8 * t4);
                qs1 = __shfl_sync(FULL, s, 8 * t4 + 4);
            }
            // The next segment's q travels while this one streams.
            Pos pn = p;
            pn.t = p.nt - 1;
            if (x + take < x_end) {
                advance(a, sh, pn);
                load_q(pn);
            }
            // The new token is the last key of the pair's last tile (none where the
            // context length was out of range and is taken as the table's).
            const bool stores = a.new_k && p.t + take == p.nt && __ldg(a.ctx_lens + p.b) == ctx;
            uint2 nk = make_uint2(0, 0), nv = nk;
            int new_blk = -1;
            if (stores) {
                nk = __ldg(a.new_k + p.b * a.new_k_stride + p.g * (Q8_D / 4) + lane);
                nv = __ldg(a.new_v + p.b * a.new_v_stride + p.g * (Q8_D / 4) + lane);
                new_blk = __ldg(a.block_tables + (int64_t)p.b * a.max_blocks + (int)((uint32_t)(ctx - 1) / (uint32_t)a.block_size));
            }
            float o[8][4];
#pragma unroll
            for (int c = 0; c < 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
            float m0 = -INFINITY, m1 = -INFINITY, mv0 = -INFINITY, mv1 = -INFINITY, l0 = 0.f, l1 = 0.f;

            for (int i = 0; i < take; ++i, ++n) {
                const int stage = n % ST;
                // (The lanes' own clocks may differ at the limit: they decide as one.)
                if (!__all_sync(FULL, mbar_wait(&bar[stage], (n / ST) & 1))) {
                    if (lane == 0) record_error(a.err, PA_DEV_TIMEOUT, 500 + warp);
                    // Let the copies already issued land before shared memory goes away.
                    for (int j = n + 1; j < issued; ++j) (void)mbar_wait(&bar[j % ST], (j / ST) & 1);
                    ok = false;
                    break;
                }
                const uint32_t ks = smem_addr(ring + stage * STAGE_BYTES), vs = ks + TILE_BYTES;
                const int nvalid = min(KT, ctx - (p.t + i) * KT);
                if (stores && i + 1 == take && new_blk >= 0 && new_blk < a.num_blocks) {
                    // (An invalid block reads as zeros, as without the fusion.)
                    const int key = nvalid - 1;  // of the tile
                    uint32_t ke, ve;
                    const uint32_t kc = quantise_row<FMT>(nk, ke), vc = quantise_row<FMT>(nv, ve);
                    const uint32_t at = (uint32_t)key * Q8_D + (uint32_t)(((lane >> 2) ^ (key & 7)) << 4) + (uint32_t)(lane & 3) * 4;
                    *reinterpret_cast<uint32_t *>(ring + stage * STAGE_BYTES + at) = kc;
                    *reinterpret_cast<uint32_t *>(ring + stage * STAGE_BYTES + TILE_BYTES + at) = vc;
                    const int64_t row = ((int64_t)new_blk * a.Hkv + p.g) * a.block_size +
                                        (int)((uint32_t)(ctx - 1) % (uint32_t)a.block_size);
                    *reinterpret_cast<uint32_t *>(a.k_codes + row * Q8_D + 4 * lane) = kc;
                    *reinterpret_cast<uint32_t *>(a.v_codes + row * Q8_D + 4 * lane) = vc;
                    if (lane == key) {
                        k_byte[0] = ke;
                        v_byte[0] = ve;
                        a.k_scales[row] = (uint8_t)ke;
                        a.v_scales[row] = (uint8_t)ve;
                    }
                    fence_proxy_async_smem();  // a later copy overwrites these bytes
                    __syncwarp();
                }
                // Lane j holds key j's scale, and the exponent of its value's.
                const float k_sc = q8_scale(k_byte[0]);
                const float v_ex = v_byte[0] == 255 ? NAN : (float)((int)v_byte[0] - 127);
                // ---- S^T = K.Q^T, 16 keys per MMA; the two chains are independent
                float s[NG][4];
#pragma unroll
                for (int u = 0; u < NG; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
#pragma unroll
                    for (int u = 0; u < NG; ++u) {
                        uint32_t r[4], a0, a1, a2, a3;
                        ldsm_x4(ks + (uint32_t)(u * 16 + (mi & 1) * 8 + r8) * Q8_D + (uint32_t)(((c + (mi >> 1)) ^ r8) << 4), r);
                        q8_to_f16<FMT>(r[0], a0, a2);
                        q8_to_f16<FMT>(r[1], a1, a3);
                        mma16816(s[u], a0, a1, a2, a3, qb[c][0], qb[c][1]);
                        q8_to_f16<FMT>(r[2], a0, a2);
                        q8_to_f16<FMT>(r[3], a1, a3);
                        mma16816(s[u], a0, a1, a2, a3, qb[c + 1][0], qb[c + 1][1]);
                    }
                }
                // ---- scores x and weighted exponents y of keys 16u + g4 (elements 0, 1)
                // and 16u + g4 + 8 (2, 3), heads 2*t4 (0, 2) and 2*t4 + 1 (1, 3)
                float xx[NG][4], yy[NG][4];
#pragma unroll
                for (int u = 0; u < NG; ++u) {
                    const int key0 = u * 16 + g4, key1 = key0 + 8;
                    const float k0 = __shfl_sync(FULL, k_sc, key0), k1 = __shfl_sync(FULL, k_sc, key1);
                    const float v0 = __shfl_sync(FULL, v_ex, key0), v1 = __shfl_sync(FULL, v_ex, key1);
                    xx[u][0] = s[u][0] * score_scale(k0, qs0);
                    xx[u][1] = s[u][1] * score_scale(k0, qs1);
                    xx[u][2] = s[u][2] * score_scale(k1, qs0);
                    xx[u][3] = s[u][3] * score_scale(k1, qs1);
                    yy[u][0] = xx[u][0] + v0;
                    yy[u][1] = xx[u][1] + v0;
                    yy[u][2] = xx[u][2] + v1;
                    yy[u][3] = xx[u][3] + v1;
                    if (nvalid < KT) {  // the context's last tile
                        if (key0 >= nvalid) xx[u][0] = xx[u][1] = yy[u][0] = yy[u][1] = -INFINITY;
                        if (key1 >= nvalid) xx[u][2] = xx[u][3] = yy[u][2] = yy[u][3] = -INFINITY;
                    }
                }
                float tx0 = -INFINITY, tx1 = -INFINITY, ty0 = -INFINITY, ty1 = -INFINITY;
#pragma unroll
                for (int u = 0; u < NG; ++u) {
                    tx0 = fmaxf(tx0, fmaxf(xx[u][0], xx[u][2]));
                    tx1 = fmaxf(tx1, fmaxf(xx[u][1], xx[u][3]));
                    ty0 = fmaxf(ty0, fmaxf(yy[u][0], yy[u][2]));
                    ty1 = fmaxf(ty1, fmaxf(yy[u][1], yy[u][3]));
                }
                const bool move =
                    (h0 && (tx0 > m0 + kLazyRescale || ty0 > mv0 + (kWeightTop + kLazyRescale))) ||
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
                // ---- O^T += V^T.P'^T; the weights become the B fragments by transposes
                uint32_t b0[NG], b1[NG];
#pragma unroll
                for (int u = 0; u < NG; ++u) {
                    l0 += fast_exp2(xx[u][0] - um0) + fast_exp2(xx[u][2] - um0);
                    l1 += fast_exp2(xx[u][1] - um1) + fast_exp2(xx[u][3] - um1);
                    b0[u] = transpose8x8(pack_f16(fast_exp2(yy[u][0] - uv0), fast_exp2(yy[u][1] - uv1)));
                    b1[u] = transpose8x8(pack_f16(fast_exp2(yy[u][2] - uv0), fast_exp2(yy[u][3] - uv1)));
                }
#pragma unroll
                for (int u = 0; u < NG; ++u) {
                    // Rows past the context may hold anything (NaN codes included) and
                    // 0 * NaN is not 0: their lanes read the row of zeros.
                    const int vk = u * 16 + (mi & 1) * 8 + r8;
                    const uint32_t vrow = vk < nvalid ? vs + (uint32_t)vk * Q8_D : zero_row;
#pragma unroll
                    for (int c = 0; c < 8; c += 2) {
                        uint32_t r[4], a0, a1, a2, a3;
                        ldsm_x4_t(vrow + (uint32_t)(((c + (mi >> 1)) ^ r8) << 4), r);
                        v_to_f16<FMT>(r[0], a0, a1);
                        v_to_f16<FMT>(r[1], a2, a3);
                        mma16816(o[c], a0, a1, a2, a3, b0[u], b1[u]);
                        v_to_f16<FMT>(r[2], a0, a1);
                        v_to_f16<FMT>(r[3], a2, a3);
                        mma16816(o[c + 1], a0, a1, a2, a3, b0[u], b1[u]);
                    }
                }
                __syncwarp();  // every lane has read the stage
#pragma unroll
                for (int j = 1; j < ST; ++j) {
                    k_byte[j - 1] = k_byte[j];
                    v_byte[j - 1] = v_byte[j];
                }
                if (ix < x_end) {
                    issue(stage, k_byte[ST - 1], v_byte[ST - 1]);
                    ++issued;
                }
            }
            if (!ok) break;
            // ---- segment end.  This lane holds dims 16c + 2*g4, +1 of heads 2*t4, 2*t4+1.
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
                l0 += __shfl_xor_sync(FULL, l0, d);
                l1 += __shfl_xor_sync(FULL, l1, d);
            }
            if (p.t == 0 && take == p.nt) {
                const OutScale f0 = out_scale(m0, mv0, l0), f1 = out_scale(m1, mv1, l1);
                __nv_bfloat16 *dst = a.out + ((int64_t)p.b * a.Hq + (int64_t)p.g * G + 2 * t4) * Q8_D + 2 * g4;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (h0) *reinterpret_cast<__nv_bfloat162 *>(dst + 16 * c) = __floats2bfloat162_rn(f0(o[c][0]), f0(o[c][2]));
                    if (h1) *reinterpret_cast<__nv_bfloat162 *>(dst + Q8_D + 16 * c) = __floats2bfloat162_rn(f1(o[c][1]), f1(o[c][3]));
                }
            } else {
                // A piece of the pair: only a range's first and last segments can be.
                const int slot = 2 * warp + (x == x_begin ? 0 : 1);
                float *piece = stash + slot * kPiece<G>;
                float *dst = piece + 2 * t4 * Q8_D + 2 * g4;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (h0) *reinterpret_cast<float2 *>(dst + 16 * c) = make_float2(o[c][0], o[c][2]);
                    if (h1) *reinterpret_cast<float2 *>(dst + Q8_D + 16 * c) = make_float2(o[c][1], o[c][3]);
                }
                if (g4 == 0) {
                    float4 *ml = reinterpret_cast<float4 *>(piece + G * Q8_D);
                    if (h0) ml[2 * t4] = make_float4(m0, mv0, l0, 0.f);
                    if (h1) ml[2 * t4 + 1] = make_float4(m1, mv1, l1, 0.f);
                }
                if (lane == 0) piece_pair[slot] = make_int2(p.b, p.g);
            }
            x += take;
            p = pn;
        }
        if (!ok && lane == 0) *abort = 1;
    }

    // ---- the CTA's pieces, pair by pair.  Lane i stands for piece i; a pair's
    // pieces are neighbours, since the warps' ranges follow the list.
    __syncthreads();
    if (*abort) return;  // a wait ran out: the call's result is void
    {
        const int2 bg = lane < 2 * NW ? piece_pair[lane] : make_int2(-1, 0);
        const unsigned valid = __ballot_sync(FULL, bg.x >= 0);
        const unsigned before = valid & ((1u << lane) - 1);
        const int from = before ? 31 - __clz(before) : 0;
        const int pb = __shfl_sync(FULL, bg.x, from), pg = __shfl_sync(FULL, bg.y, from);
        const unsigned heads = __ballot_sync(FULL, bg.x >= 0 && (!before || pb != bg.x || pg != bg.y));
        for (int item = warp; item < __popc(heads) * G; item += NW) {
            const int h = item % G;
            unsigned rest = heads;
            for (int k = item / G; k > 0; --k) rest &= rest - 1;
            const int i0 = __ffs(rest) - 1;  // the pair's first piece
            rest &= rest - 1;
            const unsigned mask = valid & ~((1u << i0) - 1) & (rest ? (1u << (__ffs(rest) - 1)) - 1 : FULL);
            const int b = __shfl_sync(FULL, bg.x, i0), g = __shfl_sync(FULL, bg.y, i0);
            const Merged r = merge_pieces<G, false>(stash, [](int j) { return j; }, mask, h);
            const uint32_t nt = cum[b + 1] - cum[b], x0 = (uint32_t)a.Hkv * cum[b] + (uint32_t)g * nt;
            const int64_t row = (int64_t)b * a.Hq + (int64_t)g * G + h;
            if (x0 >= c_begin && x0 + nt <= c_end) {
                write_out(a, r, row);
                continue;
            }
            // The pair spans CTAs: leave this head's part and count it.
            const int began = x0 >= c_begin;
            float *part = a.ws_part + ((int64_t)2 * cta + began) * kPiece<G>;
            *reinterpret_cast<float4 *>(part + h * Q8_D + 4 * lane) = r.o;
            if (lane == 0) *reinterpret_cast<float4 *>(part + G * Q8_D + 4 * h) = make_float4(r.m, r.mv, r.l, 0.f);
            __syncwarp();
            const int c0 = span[began].x, n = span[began].y;
            int last = 0;
            if (lane == 0) {
                int *cnt = a.ws_cnt + c0 * 8 + h;
                last = add_acq_rel(cnt, 1) == n - 1;
                if (last) *cnt = 0;  // ready for the next call
            }
            if (__shfl_sync(FULL, last, 0)) {
                __syncwarp();
                merge_parts<G>(a, row, c0, n, h);
            }
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
                                                   (int)kMaxSmem);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(decode_q8_kernel)");
        g_attr_done[dev][gi].store(1, std::memory_order_release);
    }
    return launch_pdl(decode_q8_kernel<G, FMT>, dim3((unsigned)grid), dim3(NT), smem_bytes(a.batch, G), st,
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

pa_status decode_q8_impl(void *out, const void *q, int64_t q_row_stride, const void *new_k, int64_t new_k_row_stride,
                         const void *new_v, int64_t new_v_row_stride, void *k_cache, void *v_cache, void *k_scale,
                         void *v_scale, const int32_t *block_tables, int32_t max_blocks_per_seq,
                         const int32_t *context_lens, int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t format,
                         float softmax_scale, void *workspace, size_t workspace_bytes, pa_stream_t stream) {
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
    // The list's units (up to three per tile) are numbered in 32 bits.
    if ((int64_t)batch * (((int64_t)max_blocks_per_seq * block_size + KT - 1) / KT) >= (1LL << 30) / num_kv_heads)
        return fail(PA_ERR_UNSUPPORTED, "batch x block-table capacity too large (%d x %lld tokens)", batch,
                    (long long)max_blocks_per_seq * block_size);
    if (q_row_stride < (int64_t)num_q_heads * Q8_D || q_row_stride % 8)
        return fail(PA_ERR_INVALID_ARG, "q_row_stride must be >= num_q_heads*head_dim and a multiple of 8");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) ||
        !aligned16(v_scale))
        return fail(PA_ERR_INVALID_ARG, "out/q/cache/scale pointers must be 16-byte aligned");
    if (!(softmax_scale > 0.f) || !isfinite(softmax_scale))
        return fail(PA_ERR_INVALID_ARG, "softmax_scale must be positive and finite");
    const size_t need = ws_bytes(G);
    if (!workspace || workspace_bytes < need)
        return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? workspace_bytes : (size_t)0);
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");

    const int box = block_size % KT ? 16 : KT;  // a TMA box stays inside a block
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
    A.new_k = static_cast<const uint2 *>(new_k);
    A.new_v = static_cast<const uint2 *>(new_v);
    A.new_k_stride = new_k_row_stride / 4;
    A.new_v_stride = new_v_row_stride / 4;
    A.k_codes = static_cast<uint8_t *>(k_cache);
    A.v_codes = static_cast<uint8_t *>(v_cache);
    A.k_scales = static_cast<uint8_t *>(k_scale);
    A.v_scales = static_cast<uint8_t *>(v_scale);
    A.ws_cnt = reinterpret_cast<int *>(ws);
    A.ws_part = reinterpret_cast<float *>(ws + kWsParts);
    A.err = device_error_ptr();
    A.checked = checked_mode() ? 1 : 0;
    const int grid = std::min(sm_count(), kMaxGrid);
    if (grid <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return format == PA_Q8_E4M3 ? launch_g<PA_Q8_E4M3>(G, A, tk, tv, grid, s)
                                : launch_g<PA_Q8_INT8>(G, A, tk, tv, grid, s);
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_decode_q8_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
    if (head_dim != pa::Q8_D || !pa::supported_group(num_q_heads, num_kv_heads)) return 0;
    return pa::ws_bytes(num_q_heads / num_kv_heads);
}

pa_status pa_decode_q8(void *out, const void *q, int64_t q_row_stride, const void *k_cache, const void *v_cache,
                       const void *k_scale, const void *v_scale, const int32_t *block_tables,
                       int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                       int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                       int32_t format, float softmax_scale, void *workspace, size_t workspace_bytes,
                       pa_stream_t stream) {
    return pa::decode_q8_impl(out, q, q_row_stride, nullptr, 0, nullptr, 0, const_cast<void *>(k_cache),
                              const_cast<void *>(v_cache), const_cast<void *>(k_scale), const_cast<void *>(v_scale),
                              block_tables, max_blocks_per_seq, context_lens, batch, num_q_heads, num_kv_heads,
                              head_dim, block_size, num_blocks, format, softmax_scale, workspace, workspace_bytes,
                              stream);
}

pa_status pa_decode_store_q8(void *out, const void *q, int64_t q_row_stride, const void *new_k,
                             int64_t new_k_row_stride, const void *new_v, int64_t new_v_row_stride, void *k_cache,
                             void *v_cache, void *k_scale, void *v_scale, const int32_t *block_tables,
                             int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t batch,
                             int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                             int32_t num_blocks, int32_t format, float softmax_scale, void *workspace,
                             size_t workspace_bytes, pa_stream_t stream) {
    using namespace pa;
    if (batch > 0) {
        if (!new_k || !new_v) return fail(PA_ERR_INVALID_ARG, "null new_k/new_v");
        if (!aligned16(new_k) || !aligned16(new_v)) return fail(PA_ERR_INVALID_ARG, "new_k/new_v must be 16-byte aligned");
        const int64_t row = (int64_t)num_kv_heads * Q8_D;
        if (new_k_row_stride < row || new_v_row_stride < row || new_k_row_stride % 8 || new_v_row_stride % 8)
            return fail(PA_ERR_INVALID_ARG, "new_k/new_v row strides must be >= num_kv_heads*head_dim and multiples of 8");
    }
    return decode_q8_impl(out, q, q_row_stride, new_k, new_k_row_stride, new_v, new_v_row_stride, k_cache, v_cache,
                          k_scale, v_scale, block_tables, max_blocks_per_seq, context_lens, batch, num_q_heads,
                          num_kv_heads, head_dim, block_size, num_blocks, format, softmax_scale, workspace,
                          workspace_bytes, stream);
}

}  // extern "C"
