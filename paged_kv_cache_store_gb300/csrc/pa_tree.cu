// pa_tree.cu -- attention of a tree of drafted tokens over the paged pool.
//
// What it computes: sequence b has ctx keys, its n drafted tokens the last of
// them.  Draft i, head h attends to the ctx - n keys before the drafts and to
// draft j where bit j of its mask is set:
//   s_p = scale <q, K_p>,  out = sum_p softmax(s)_p V_p  over the keys it sees.
//
// How: the n drafts of the G query heads of one kv head are up to 64 * 8 rows
// over the same keys, so every K/V byte is used by all of them and the scores are
// a matrix product for the 5th-generation tensor cores.  An item is one
// (sequence, kv head, block of 128 * NT rows); its 64-key tiles, laid end to end
// over all items, are cut into one range of equal cost per CTA.  Roles of a CTA:
//   warp 0     K and V tiles by TMA into rings of ST stages, block ids 32 at a time
//   warp 1     S = Q K^T (M = 128, N = 64, K = 128) into one of two TMEM buffers
//   warp 2     O += P V (P from TMEM, V as an MN-major operand)
//   warp 3     Q rows of the next item into shared memory
//   warps 4..  one thread per row: online softmax in base 2, P over S as bf16
// Of the 128 rows of an MMA only the live ones are loaded and read back; the
// others hold whatever the memory held, which cannot reach a live row.
//
// An item cut between CTAs leaves (m, l, o) in fp32 in the workspace; the warp
// that arrives last at its 32 rows combines the parts in order.
//
// l is summed from the rounded P that the product uses, so that the weights sum
// to one as they are.
//
// What a mask hides may be anything: scores are replaced before the maximum,
// and a draft's V values that are not finite are taken out of the tile (0 times
// such a value would be NaN in every row) and added to the rows that see them.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int D = 128;
constexpr int TILE = 64;                 // keys per tile
constexpr int ROWS = 128;                // rows of one MMA
constexpr int KV_BYTES = TILE * D * 2;   // a K or V tile: 16 KiB, [2 halves][64 rows][128 B]
constexpr int KV_HALF = KV_BYTES / 2;
constexpr int QTILE = ROWS * D * 2;      // 32 KiB, [2 halves][128 rows][128 B]
constexpr int QHALF = QTILE / 2;
constexpr uint32_t SBO = 1024;           // 8 rows x 128 B between core-matrix groups
constexpr uint32_t IDESC_S = idesc_bf16_f32(ROWS, TILE, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(ROWS, D, false, true);
constexpr int kMaxBatch = 2048;
constexpr int kMaxDrafts = 64;
constexpr int kMaxGrid = 256;
constexpr int kItemCost = 1;             // an item costs this many tiles on top of its own
constexpr int kMinTiles = 2;             // a CTA's share at least
constexpr float kLazy = 8.f;             // log2 headroom before the running maximum must move
constexpr unsigned FULL = 0xffffffffu;

template <int NT>
struct Cfg {
    static constexpr int ST = NT == 1 ? 5 : 4;  // ring stages
    static constexpr int THREADS = 128 + 128 * NT;
    static constexpr int OFF_K = NT * QTILE;
    static constexpr int OFF_V = OFF_K + ST * KV_BYTES;
    static constexpr int OFF_BAR = OFF_V + ST * KV_BYTES;
    // Barriers: rings, then per row tile and buffer.
    static constexpr int KFULL = 0, KEMPTY = ST, VFULL = 2 * ST, VEMPTY = 3 * ST, SFULL = 4 * ST, PFULL = SFULL + 2 * NT,
                         PDONE = PFULL + 2 * NT, OEMPTY = PDONE + 2 * NT, QFULL = OEMPTY + NT, QEMPTY = QFULL + 1,
                         DRAIN = QEMPTY + 1, NBAR = DRAIN + 2;
    static constexpr int OFF_MISC = OFF_BAR + (NBAR * 8 + 15) / 16 * 16;  // TMEM address, abort flag, marks, scan scratch
    static constexpr int OFF_ARR = OFF_MISC + 128;       // ctx, n, cum [batch + 1]
    static constexpr uint32_t COLS = NT == 1 ? 256 : 512;
    static constexpr uint32_t COL_O = NT * 128;          // S(h, b) at h * 128 + b * 64, O(h) at COL_O + h * 128
};
__host__ __device__ constexpr size_t tree_smem(int off_arr, int batch) { return off_arr + 12 * (size_t)(batch + 1) + 1024; }
static_assert(tree_smem(Cfg<1>::OFF_ARR, kMaxBatch) <= 232448 && tree_smem(Cfg<2>::OFF_ARR, kMaxBatch) <= 232448,
              "shared memory");

// Floats of a part: o [rows][D], (m, l) [rows], a multiple of 16 bytes.
__host__ __device__ constexpr size_t slot_of(int rows) { return ((size_t)rows * (D + 2) + 3) / 4 * 4; }

struct TreeArgs {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const __nv_bfloat16 *v_cache;
    int64_t q_stride;  // elements between tokens
    const int32_t *bt, *ctx, *lens;
    const unsigned long long *mask;  // null: a chain
    int32_t max_blocks, batch, drafts, Hq, Hkv, G, block_size, num_blocks, box_rows, checked;
    float scale_log2;
    int *count;    // [grid][8] arrivals
    float *parts;  // [grid][2] of slot_of(part_rows)
    int32_t part_rows;
    DevError *err;
};

__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort, DevError *err,
                                              int where) {
    if (mbar_try_wait(smem_addr(bar), parity)) return true;
    if (*abort) return false;
    if (mbar_wait(bar, parity)) return true;
    record_error(err, PA_DEV_TIMEOUT, where);
    *abort = 1;
    return false;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
// 1 where a bf16 half of the word is NaN or infinite (its exponent all ones).
__device__ __forceinline__ bool not_finite2(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// Where a CTA's range stands: an item and the tiles of it that are the CTA's.
struct Seg {
    int b, g, blk;       // sequence, kv head, row block
    int t0, t1, nt;      // tiles [t0, t1) of nt
    int rows;            // live rows of the item
    uint32_t first;      // the item's first unit
};

template <int NT>
struct Walker {
    const int *ctx_s, *n_s;
    const uint32_t *cum;
    int G;
    uint32_t x, x1;
    int b;
    __device__ __forceinline__ int rows_of(int bb) const { return n_s[bb] * G; }
    __device__ __forceinline__ int tiles_of(int bb) const { return (ctx_s[bb] + TILE - 1) / TILE; }
    __device__ __forceinline__ void start(uint32_t x0, uint32_t xe, int batch) {
        x = x0;
        x1 = xe;
        int lo = 0, hi = batch - 1;  // the last b with cum[b] <= x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cum[mid] <= x) lo = mid; else hi = mid - 1;
        }
        b = lo;
    }
    // The next item that has tiles in the range.
    __device__ __forceinline__ bool next(Seg &s) {
        while (x < x1) {
            while (cum[b + 1] <= x) ++b;
            const int nt = tiles_of(b), u = nt + kItemCost;
            const int blocks = (rows_of(b) + ROWS * NT - 1) / (ROWS * NT);
            const uint32_t local = x - cum[b], it = local / (uint32_t)u;
            const int t0 = (int)(local - it * (uint32_t)u);
            const uint32_t first = cum[b] + it * (uint32_t)u;
            const uint32_t end = min(first + (uint32_t)u, x1);
            x = end;
            if (t0 >= nt) continue;
            s.b = b;
            s.g = (int)it / blocks;
            s.blk = (int)it % blocks;
            s.t0 = t0;
            s.t1 = min((int)(end - first), nt);
            s.nt = nt;
            s.rows = min(rows_of(b) - s.blk * ROWS * NT, ROWS * NT);
            s.first = first;
            return true;
        }
        return false;
    }
};

template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::THREADS, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                       const __grid_constant__ TreeArgs a) {
    using C = Cfg<NT>;
    constexpr int ST = C::ST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    uint32_t *wsum = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC + 16);
    int *ctx_s = reinterpret_cast<int *>(smem + C::OFF_ARR);
    int *n_s = ctx_s + (a.batch + 1);
    uint32_t *cum = reinterpret_cast<uint32_t *>(n_s + (a.batch + 1));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int NWARPS = C::THREADS / 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NBAR; ++i) {
            const bool per_warp = (i >= C::PFULL && i < C::PFULL + 2 * NT) || (i >= C::OEMPTY && i < C::OEMPTY + NT);
            mbar_init(&bar[i], per_warp ? 4u : 1u);  // the four softmax warps of a row tile arrive one each
        }
        abort[0] = abort[1] = abort[2] = 0;  // and the two marks behind it
        fence_mbar_init();
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::COLS);
        tmem_relinquish();
    }
    pdl_wait_then_release();
    // Lengths, and the running sum of the sequences' units (tiles, and kItemCost
    // more per item).
    uint32_t carry = 0;
    for (int base = 0; base < a.batch; base += C::THREADS) {
        const int b = base + threadIdx.x;
        uint32_t u = 0;
        if (b < a.batch) {
            int ctx = __ldg(a.ctx + b);
            int n = a.lens ? __ldg(a.lens + b) : min(a.drafts, max(ctx, 0));
            if (ctx < 0 || ctx > (int64_t)a.max_blocks * a.block_size || n < 0 || n > a.drafts || n > ctx ||
                (!a.lens && ctx > 0 && ctx < a.drafts)) {
                if (blockIdx.x == 0) record_error(a.err, PA_DEV_BAD_CONTEXT, b);
                n = 0;
            }
            if (n == 0) ctx = 0;
            ctx_s[b] = ctx;
            n_s[b] = n;
            const int blocks = (n * a.G + ROWS * NT - 1) / (ROWS * NT);
            u = n ? (uint32_t)((ctx + TILE - 1) / TILE + kItemCost) * (uint32_t)(a.Hkv * blocks) : 0u;
        }
        uint32_t inc = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(FULL, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        uint32_t before = carry, all = carry;
        for (int w = 0; w < NWARPS; ++w) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        if (b < a.batch) cum[b] = before + inc - u;
        carry = all;
        __syncthreads();
    }
    if (threadIdx.x == 0) cum[a.batch] = carry;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t P = carry;  // units in all
    const uint32_t nC = min((uint32_t)gridDim.x, max(1u, P / kMinTiles));
    Walker<NT> walk{ctx_s, n_s, cum, a.G};
    const bool works = blockIdx.x < nC && P > 0;
    if (works) {
        walk.start((uint32_t)((uint64_t)blockIdx.x * P / nC), (uint32_t)((uint64_t)(blockIdx.x + 1) * P / nC), a.batch);
    } else {
        walk.x = walk.x1 = 0;
        walk.b = 0;
    }
    // The CTA whose range holds unit x.
    auto owner = [&](uint32_t x) -> int { return (int)(((uint64_t)(x + 1) * nC - 1) / P); };
    Seg s;
    bool ok = true;

    if (warp == 0) {
        // ---------------------------------------------------------------- K and V tiles
        uint32_t gg = 0;
        const int R = a.box_rows;
        while (ok && walk.next(s)) {
            const int32_t *bt = a.bt + (int64_t)s.b * a.max_blocks;
            const int key_end = ctx_s[s.b];
            const int last = (key_end - 1) / a.block_size;  // the sequence's last block
            int base = s.t0 * TILE / a.block_size;
            int id = __ldg(bt + min(base + lane, last));    // block ids base + lane
            for (int j = s.t0; ok && j < s.t1; ++j, ++gg) {
                const int st = gg % ST;
                const int nsub = (min(TILE, key_end - j * TILE) + R - 1) / R;
                if (lane == 0) {
                    ok = wait_or_abort(&bar[C::KEMPTY + st], ((gg / ST) & 1u) ^ 1u, abort, a.err, 700) &&
                         wait_or_abort(&bar[C::VEMPTY + st], ((gg / ST) & 1u) ^ 1u, abort, a.err, 701);
                    if (ok) {
                        mbar_arrive_expect_tx(&bar[C::KFULL + st], (uint32_t)(nsub * R * D * 2));
                        mbar_arrive_expect_tx(&bar[C::VFULL + st], (uint32_t)(nsub * R * D * 2));
                    }
                }
                ok = __shfl_sync(FULL, ok ? 1 : 0, 0) != 0;
                for (int sub = 0; ok && sub < nsub; ++sub) {
                    const int key = j * TILE + sub * R, lb = key / a.block_size;
                    if (lb >= base + 32) {
                        base = lb;
                        id = __ldg(bt + min(base + lane, last));
                    }
                    const int blk = __shfl_sync(FULL, id, lb - base);
                    if (lane == 0) {
                        const bool bad = blk < 0 || blk >= a.num_blocks;
                        if (bad && a.checked)
                            record_error(a.err, PA_DEV_BAD_BLOCK, (long long)s.b * a.max_blocks + lb);
                        // A box outside the pool is filled with zeros.
                        const int row = bad ? -2 * R : blk * a.block_size + key % a.block_size;
                        uint8_t *k = smem + C::OFF_K + st * KV_BYTES + sub * R * 128;
                        uint8_t *v = smem + C::OFF_V + st * KV_BYTES + sub * R * 128;
                        if (R == TILE) {
                            tma_load_4d_plain(k, &tmk, 0, row, 0, s.g, &bar[C::KFULL + st]);
                            tma_load_4d_plain(v, &tmv, 0, row, 0, s.g, &bar[C::VFULL + st]);
                        } else {
                            tma_load_4d_plain(k, &tmk, 0, row, 0, s.g, &bar[C::KFULL + st]);
                            tma_load_4d_plain(k + KV_HALF, &tmk, 0, row, 1, s.g, &bar[C::KFULL + st]);
                            tma_load_4d_plain(v, &tmv, 0, row, 0, s.g, &bar[C::VFULL + st]);
                            tma_load_4d_plain(v + KV_HALF, &tmv, 0, row, 1, s.g, &bar[C::VFULL + st]);
                        }
                    }
                }
                if (!ok) break;
            }
        }
        if (lane == 0 && !ok) {  // issued copies land before the shared memory is given back
            for (uint32_t x = gg >= (uint32_t)ST ? gg - ST : 0; x < gg; ++x) {
                (void)mbar_wait(&bar[C::KFULL + x % ST], (x / ST) & 1u);
                (void)mbar_wait(&bar[C::VFULL + x % ST], (x / ST) & 1u);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- S = Q K^T
        if (lane == 0) {
            uint32_t gg = 0, ui = 0, th[NT] = {};  // tiles in all, items, tiles of each row tile
            bool issued = false;
            while (ok && walk.next(s)) {
                if (!(ok = wait_or_abort(&bar[C::QFULL], ui & 1u, abort, a.err, 702))) break;
                const int nh = NT == 1 ? 1 : (s.rows + ROWS - 1) / ROWS;
                for (int j = s.t0; ok && j < s.t1; ++j, ++gg) {
                    const int st = gg % ST;
                    if (!(ok = wait_or_abort(&bar[C::KFULL + st], (gg / ST) & 1u, abort, a.err, 703))) break;
                    const uint64_t kdesc = smem_desc_sw128(smem_addr(smem + C::OFF_K + st * KV_BYTES), 16, SBO);
#pragma unroll
                    for (int h = 0; h < NT; ++h) {
                        if (h >= nh) break;
                        const int b = th[h] & 1;
                        // The buffer is free once the P.V of two tiles ago has read it.
                        if (!(ok = wait_or_abort(&bar[C::PDONE + 2 * h + b], ((th[h] >> 1) & 1u) ^ 1u, abort, a.err,
                                                 704)))
                            break;
                        tc_fence_after();
                        const uint64_t qdesc = smem_desc_sw128(smem_addr(smem + h * QTILE), 16, SBO);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_bf16_ss(tmem + h * 128 + b * TILE,
                                        qdesc + (uint64_t)(((kk >> 2) * QHALF + (kk & 3) * 32) >> 4),
                                        kdesc + (uint64_t)(((kk >> 2) * KV_HALF + (kk & 3) * 32) >> 4), IDESC_S,
                                        kk > 0 ? 1u : 0u);
                        mma_commit(&bar[C::SFULL + 2 * h + b]);
                        issued = true;
                        ++th[h];
                    }
                    if (!ok) break;
                    mma_commit(&bar[C::KEMPTY + st]);
                }
                if (ok) mma_commit(&bar[C::QEMPTY]);  // every product of the item has read Q
                ++ui;
            }
            if (issued && *abort) {
                mma_commit(&bar[C::DRAIN]);
                (void)mbar_wait(&bar[C::DRAIN], 0);
            }
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- O += P V
        if (lane == 0) {
            uint32_t gg = 0, th[NT] = {}, uh[NT] = {};
            bool issued = false;
            while (ok && walk.next(s)) {
                const int nh = NT == 1 ? 1 : (s.rows + ROWS - 1) / ROWS;
                for (int j = s.t0; ok && j < s.t1; ++j, ++gg) {
                    const int st = gg % ST;
                    if (!(ok = wait_or_abort(&bar[C::VFULL + st], (gg / ST) & 1u, abort, a.err, 705))) break;
                    const int steps = (min(TILE, ctx_s[s.b] - j * TILE) + 15) / 16;  // keys past the last: P is 0
                    const uint64_t vdesc = smem_desc_sw128(smem_addr(smem + C::OFF_V + st * KV_BYTES), KV_HALF, SBO);
#pragma unroll
                    for (int h = 0; h < NT; ++h) {
                        if (h >= nh) break;
                        const int b = th[h] & 1;
                        if (j == s.t0) {  // O is free once the last item's was read
                            if (!(ok = wait_or_abort(&bar[C::OEMPTY + h], (uh[h] & 1u) ^ 1u, abort, a.err, 706))) break;
                            ++uh[h];
                        }
                        if (!(ok = wait_or_abort(&bar[C::PFULL + 2 * h + b], (th[h] >> 1) & 1u, abort, a.err, 707)))
                            break;
                        tc_fence_after();
                        for (int kk = 0; kk < steps; ++kk)  // 16 keys a step = 8 TMEM columns of P
                            mma_bf16_ts(tmem + C::COL_O + h * 128, tmem + h * 128 + b * TILE + kk * 8,
                                        vdesc + (uint64_t)((kk * 16 * 128) >> 4), IDESC_PV,
                                        (j > s.t0 || kk > 0) ? 1u : 0u);
                        mma_commit(&bar[C::PDONE + 2 * h + b]);
                        issued = true;
                        ++th[h];
                    }
                    if (!ok) break;
                    mma_commit(&bar[C::VEMPTY + st]);
                }
            }
            if (issued && *abort) {
                mma_commit(&bar[C::DRAIN + 1]);
                (void)mbar_wait(&bar[C::DRAIN + 1], 0);
            }
        }
    } else if (warp == 3) {
        // ---------------------------------------------------------------- Q rows
        uint32_t ui = 0;
        while (ok && walk.next(s)) {
            ok = __all_sync(FULL, wait_or_abort(&bar[C::QEMPTY], (ui & 1u) ^ 1u, abort, a.err, 708));
            if (!ok) break;
            const __nv_bfloat16 *q = a.q + (int64_t)s.b * a.drafts * a.q_stride + (int64_t)s.g * a.G * D;
            const uint32_t qs = smem_addr(smem);
            const int c = lane & 15;  // two rows a step, 16 lanes each; 8 steps in flight
            for (int r0 = 0; r0 < s.rows; r0 += 16) {
                uint4 v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = r0 + 2 * e + (lane >> 4), rr = s.blk * ROWS * NT + r;
                    if (r < s.rows)
                        v[e] = __ldg(reinterpret_cast<const uint4 *>(q + (int64_t)(rr / a.G) * a.q_stride + (rr % a.G) * D) + c);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = r0 + 2 * e + (lane >> 4);
                    if (r < s.rows)
                        st_shared_u4(qs + (uint32_t)((r >> 7) * QTILE + (c >> 3) * QHALF + (r & 127) * 128 +
                                                     (((c & 7) ^ (r & 7)) << 4)),
                                     v[e]);
                }
            }
            fence_proxy_async_smem();  // the MMA reads Q through the async proxy
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[C::QFULL]);
            ++ui;
        }
    } else {
        // ---------------------------------------------------------------- softmax, output
        const int h = NT == 1 ? 0 : (warp - 4) >> 2;  // row tile
        const int quarter = warp & 3;
        const int wrow = quarter * 32, row = wrow + lane;  // row of the tile == TMEM lane
        const uint32_t t_lane = tmem + ((uint32_t)wrow << 16);
        const uint32_t t_o = t_lane + C::COL_O + h * 128;
        const float sl = a.scale_log2;
        auto wwait = [&](uint64_t *bb, uint32_t parity, int where) -> bool {
            return __all_sync(FULL, wait_or_abort(bb, parity, abort, a.err, where));
        };
        {
            // Rows past a sequence's drafts: zeros.
            const int sw = (warp - 4) + 4 * NT * blockIdx.x, nsw = 4 * NT * gridDim.x;
            const int per = a.Hq * (D / 8) ;  // 16-byte chunks of a token
            for (int t = sw; t < a.batch * a.drafts; t += nsw) {
                const int b = t / a.drafts;
                if (t - b * a.drafts < n_s[b]) continue;
                uint4 *dst = reinterpret_cast<uint4 *>(a.out) + (int64_t)t * per;
                for (int c = lane; c < per; c += 32) dst[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        // odd[seg & 1] == seg + 1: a draft's V in segment number seg held something
        // not finite.  (No warp is more than one segment ahead of another: a
        // segment's last product needs the P of all of them.)
        volatile int *odd = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 8);
        uint32_t gg = 0, th = 0;  // tiles in all (V ring), tiles of this row tile
        for (int seg = 0; ok && walk.next(s); ++seg) {
            const int live = min(max(s.rows - h * ROWS, 0), ROWS);  // live rows of this row tile
            if (live == 0) {
                gg += s.t1 - s.t0;
                continue;
            }
            const int ctx = ctx_s[s.b], n = n_s[s.b], first = ctx - n;
            const int grow = s.blk * ROWS * NT + h * ROWS + row;  // row of the (sequence, kv head)
            const int di = grow / a.G;                            // its draft
            const bool mine = row < live, wlive = wrow < live;
            unsigned long long m64 = 0;
            if (mine) {
                m64 = a.mask ? __ldg(a.mask + (int64_t)s.b * a.drafts + di) : di >= 63 ? ~0ull : (2ull << di) - 1;
                if (n < 64) m64 &= (1ull << n) - 1;
            }
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = s.t0; ok && j < s.t1; ++j, ++gg, ++th) {
                const int b = th & 1, kb = j * TILE;
                const uint32_t cs = t_lane + h * 128 + b * TILE;
                if (kb + TILE > first) {
                    // A tile with drafts: V's rows past the last key that the
                    // product reads become zeros, and drafts' values that are not
                    // finite too.  Each row tile of the item does it before its
                    // product; what the first has mended, the second leaves.
                    const int st = gg % ST;
                    if (!(ok = wwait(&bar[C::VFULL + st], (gg / ST) & 1u, 709))) break;
                    const int kend = min(TILE, ctx - kb), kpad = (kend + 15) & ~15, k0 = max(0, first - kb);
                    const uint32_t vb = smem_addr(smem + C::OFF_V + st * KV_BYTES);
                    for (int i = threadIdx.x & 127; i < (kpad - k0) * 16; i += 128) {
                        const int r = k0 + (i >> 4), c = i & 15;
                        const uint32_t at = vb + (uint32_t)((c >> 3) * KV_HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                        const uint4 w = ld_shared_v4(at);
                        if (r >= kend) {
                            if (w.x | w.y | w.z | w.w) st_shared_u4(at, make_uint4(0u, 0u, 0u, 0u));
                        } else if (not_finite2(w.x) || not_finite2(w.y) || not_finite2(w.z) || not_finite2(w.w)) {
                            // Seen by every warp at the segment's end: its P follows this.
                            odd[seg & 1] = seg + 1;
                            __threadfence_block();
                            st_shared_u4(at, make_uint4(finite_only(w.x), finite_only(w.y), finite_only(w.z),
                                                        finite_only(w.w)));
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (!(ok = wwait(&bar[C::SFULL + 2 * h + b], (th >> 1) & 1u, 710))) break;
                tc_fence_after();
                if (wlive) {
                    uint32_t r[TILE];
                    tmem_ld32(cs, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
                    tmem_ld32(cs + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
                    tmem_ld_wait();
                    if (kb + TILE > first) {
                        const int d = first - kb;  // keys of the tile before the drafts
                        unsigned long long vis;
                        if (d >= TILE) vis = ~0ull;
                        else if (d > 0) vis = ((1ull << d) - 1) | (m64 << d);
                        else vis = -d < 64 ? m64 >> -d : 0ull;
                        const uint32_t vlo = (uint32_t)vis, vhi = (uint32_t)(vis >> 32);
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            if (!((vlo >> k) & 1u)) r[k] = __float_as_uint(-INFINITY);
                            if (!((vhi >> k) & 1u)) r[k + 32] = __float_as_uint(-INFINITY);
                        }
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k2 = 0; k2 < TILE / 2; ++k2)
                        m4[k2 & 3] = max3(m4[k2 & 3], __uint_as_float(r[2 * k2]), __uint_as_float(r[2 * k2 + 1]));
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    const bool grow_m = mine && (mx - m_run) * sl > kLazy;  // rows that are not live stay put
                    const float m_new = grow_m ? mx : m_run;
                    const float alpha = grow_m ? fast_exp2((m_run - m_new) * sl) : 1.f;
                    if (j > s.t0 && __any_sync(FULL, grow_m)) {
                        // O holds the products up to the previous tile before it is rescaled.
                        if (!(ok = wwait(&bar[C::PDONE + 2 * h + ((th - 1) & 1)], ((th - 1) >> 1) & 1u, 711))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t o[32];
                            tmem_ld32(t_o + c * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(t_o + c * 32, o);
                        }
                    }
                    l_run *= alpha;
                    m_run = m_new;
                    const float neg_m = m_run == -INFINITY ? 0.f : -m_run * sl;
                    float rs[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t pk[TILE / 2];
#pragma unroll
                    for (int k2 = 0; k2 < TILE / 2; ++k2) {
                        const float p0 = fast_exp2(fmaf(__uint_as_float(r[2 * k2]), sl, neg_m));
                        const float p1 = fast_exp2(fmaf(__uint_as_float(r[2 * k2 + 1]), sl, neg_m));
                        pk[k2] = pack_bf16(p0, p1);
                        rs[k2 & 3] += bf16lo(pk[k2]) + bf16hi(pk[k2]);
                    }
                    tmem_st32(cs, pk);  // P over the first 32 columns of the buffer
                    tmem_st_wait();
                    l_run += (rs[0] + rs[1]) + (rs[2] + rs[3]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[C::PFULL + 2 * h + b]);
            }
            if (!ok) break;
            // ---- the segment's rows
            if (!(ok = wwait(&bar[C::PDONE + 2 * h + ((th - 1) & 1)], ((th - 1) >> 1) & 1u, 712))) break;
            tc_fence_after();
            uint32_t o[D];
            if (wlive) {
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_o + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[32 * c]));
                tmem_ld_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[C::OEMPTY + h]);
            if (!wlive) continue;
            if (odd[seg & 1] == seg + 1) {
                // What was taken out of V: added to the rows that see it.
                const int lo = max(0, s.t0 * TILE - first), hi = min(n, s.t1 * TILE - first);  // drafts of the segment
                for (int j = lo; j < hi; ++j) {
                    const int p = first + j, blk = __ldg(a.bt + (int64_t)s.b * a.max_blocks + p / a.block_size);
                    if (blk < 0 || blk >= a.num_blocks) continue;
                    const uint2 *v = reinterpret_cast<const uint2 *>(
                        a.v_cache + (((int64_t)blk * a.block_size + p % a.block_size) * a.Hkv + s.g) * D);
                    const uint2 w = __ldg(v + lane);  // the row across the warp
                    if (!__any_sync(FULL, not_finite2(w.x) || not_finite2(w.y))) continue;
                    const bool sees = mine && ((m64 >> j) & 1);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const uint32_t w0 = __shfl_sync(FULL, w.x, c), w1 = __shfl_sync(FULL, w.y, c);
                        const float x[4] = {bf16lo(w0), bf16hi(w0), bf16lo(w1), bf16hi(w1)};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (sees && !isfinite(x[e])) o[4 * c + e] = __float_as_uint(__uint_as_float(o[4 * c + e]) + x[e]);
                    }
                }
            }
            const bool whole = s.t0 == 0 && s.t1 == s.nt;
            auto out_row = [&](int gr) -> __nv_bfloat16 * {
                return a.out + (((int64_t)s.b * a.drafts + gr / a.G) * a.Hq + s.g * a.G + gr % a.G) * D;
            };
            if (whole) {
                if (mine) {
                    const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // a row that sees nothing: zeros
                    uint4 *dst = reinterpret_cast<uint4 *>(out_row(grow));
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const uint32_t *v = &o[8 * c];
                        dst[c] = make_uint4(pack_bf16(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv),
                                            pack_bf16(__uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv),
                                            pack_bf16(__uint_as_float(v[4]) * inv, __uint_as_float(v[5]) * inv),
                                            pack_bf16(__uint_as_float(v[6]) * inv, __uint_as_float(v[7]) * inv));
                    }
                }
                continue;
            }
            // A part: slot 1 of the item's first CTA, slot 0 of the others.
            const int c0 = owner(s.first), nparts = owner(s.first + (uint32_t)s.nt - 1) - c0 + 1;
            const size_t slot_floats = slot_of(a.part_rows);
            const int trow = h * ROWS + row;
            {
                float *slot = a.parts + (size_t)(2 * blockIdx.x + (blockIdx.x == c0 ? 1 : 0)) * slot_floats;
                if (mine) {
                    float4 *dst = reinterpret_cast<float4 *>(slot + (size_t)trow * D);
#pragma unroll
                    for (int c = 0; c < D / 4; ++c)
                        dst[c] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                             __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
                    reinterpret_cast<float2 *>(slot + (size_t)a.part_rows * D)[trow] = make_float2(m_run * sl, l_run);
                }
            }
            __threadfence();
            __syncwarp();
            int arrived = 0;
            int *cnt = a.count + c0 * 8 + h * 4 + quarter;
            if (lane == 0) arrived = atomicAdd(cnt, 1);
            arrived = __shfl_sync(FULL, arrived, 0);
            if (arrived != nparts - 1) continue;
            __threadfence();
            if (lane == 0) *cnt = 0;  // as it was found
            for (int rr = 0; rr < min(32, live - wrow); ++rr) {
                const int tr = h * ROWS + wrow + rr;
                float m = -INFINITY, l = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int p = 0; p < nparts; ++p) {
                    const float *slot = a.parts + (size_t)(2 * (c0 + p) + (p == 0 ? 1 : 0)) * slot_floats;
                    const float2 ml = __ldcg(reinterpret_cast<const float2 *>(slot + (size_t)a.part_rows * D) + tr);
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(slot + (size_t)tr * D) + lane);
                    const float mn = fmaxf(m, ml.x);
                    if (mn == -INFINITY) {  // nothing seen so far; NaN goes on
                        acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
                        l += ml.y;
                        continue;
                    }
                    const float f0 = fast_exp2(m - mn), f1 = fast_exp2(ml.x - mn);
                    acc.x = acc.x * f0 + v.x * f1;
                    acc.y = acc.y * f0 + v.y * f1;
                    acc.z = acc.z * f0 + v.z * f1;
                    acc.w = acc.w * f0 + v.w * f1;
                    l = l * f0 + ml.y * f1;
                    m = mn;
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint2 w = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                reinterpret_cast<uint2 *>(out_row(s.blk * ROWS * NT + tr))[lane] = w;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::COLS);
}

// Counters, then the parts.  A row block of an item has at most min(drafts * G,
// 128 * NT) rows.
struct Layout {
    int nt, part_rows;
    size_t parts, bytes;
};
Layout layout_of(int drafts, int G) {
    Layout l;
    l.nt = drafts * G > ROWS ? 2 : 1;
    l.part_rows = std::min(drafts * G, ROWS * l.nt);
    l.parts = (size_t)kMaxGrid * 8 * sizeof(int);
    l.bytes = l.parts + (size_t)kMaxGrid * 2 * slot_of(l.part_rows) * sizeof(float);
    return l;
}

// Per (device, variant): the shared-memory attribute has been set.
std::atomic<int> g_attr_done[64][2];

template <int NT>
pa_status launch_tree(const CUtensorMap &tmk, const CUtensorMap &tmv, const TreeArgs &a, int grid, cudaStream_t stream) {
    const size_t smem = tree_smem(Cfg<NT>::OFF_ARR, a.batch);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= 64) return fail(PA_ERR_UNSUPPORTED, "device %d", dev);
    if (!g_attr_done[dev][NT - 1].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(decode_tree_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)tree_smem(Cfg<NT>::OFF_ARR, kMaxBatch));
        if (e != cudaSuccess) return cuda_fail(e, "decode_tree_kernel shared memory");
        g_attr_done[dev][NT - 1].store(1, std::memory_order_release);
    }
    return launch_pdl(decode_tree_kernel<NT>, dim3((unsigned)grid), dim3(Cfg<NT>::THREADS), smem, stream,
                      "decode_tree_kernel", tmk, tmv, a);
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_decode_tree_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_drafts) {
    using namespace pa;
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || head_dim != D || num_drafts <= 0 ||
        num_drafts > kMaxDrafts)
        return 0;
    const int G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return 0;
    return layout_of(num_drafts, G).bytes;
}

pa_status pa_decode_tree(void *out, const void *q, int64_t q_row_stride, const void *k_cache, const void *v_cache,
                         const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
                         const int32_t *draft_lens, const int64_t *tree_mask, int32_t batch, int32_t num_drafts,
                         int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                         int32_t num_blocks, float softmax_scale, void *workspace, size_t workspace_bytes,
                         pa_stream_t stream) {
    using namespace pa;
    if (batch < 0) return fail(PA_ERR_INVALID_ARG, "batch < 0");
    if (num_drafts <= 0) return fail(PA_ERR_INVALID_ARG, "num_drafts must be positive");
    if (batch == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads)
        return fail(PA_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
    if (head_dim != D) return fail(PA_ERR_UNSUPPORTED, "head_dim %d (only 128)", head_dim);
    const int G = num_q_heads / num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return fail(PA_ERR_UNSUPPORTED, "%d query heads per kv head", G);
    if (num_drafts > kMaxDrafts) return fail(PA_ERR_UNSUPPORTED, "%d drafts (at most %d)", num_drafts, kMaxDrafts);
    if (batch > kMaxBatch) return fail(PA_ERR_UNSUPPORTED, "batch %d (at most %d)", batch, kMaxBatch);
    if (block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "block_size, max_blocks_per_seq and num_blocks must be positive");
    if (block_size % 16) return fail(PA_ERR_UNSUPPORTED, "block_size %d (a multiple of 16)", block_size);
    if ((int64_t)num_blocks * block_size > 0x7fffffffLL - 4096)
        return fail(PA_ERR_UNSUPPORTED, "num_blocks * block_size must fit 31 bits");
    const int64_t row = (int64_t)num_q_heads * D;
    if (q_row_stride < row || q_row_stride % 8)
        return fail(PA_ERR_INVALID_ARG, "q_row_stride must be >= num_q_heads*head_dim and a multiple of 8");
    if (!(softmax_scale > 0.f) || isinf(softmax_scale)) return fail(PA_ERR_INVALID_ARG, "softmax_scale must be positive");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(tree_mask) & 7u) return fail(PA_ERR_INVALID_ARG, "tree_mask must be 8-byte aligned");
    const Layout l = layout_of(num_drafts, G);
    const int64_t keys = (int64_t)max_blocks_per_seq * block_size;
    if (keys > 0x7fffffffLL - 4096) return fail(PA_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size must fit 31 bits");
    const int64_t blocks = (num_drafts * G + ROWS * l.nt - 1) / (ROWS * l.nt);
    const int64_t a_seq = (int64_t)num_kv_heads * blocks * ((keys + TILE - 1) / TILE + kItemCost);
    if (num_kv_heads > (1 << 16) || a_seq > 0x7fffffffLL / batch)
        return fail(PA_ERR_UNSUPPORTED, "too many tiles (batch * num_kv_heads * max_blocks_per_seq * block_size)");
    if (!workspace || workspace_bytes < l.bytes)
        return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0, l.bytes);
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    const int sms = sm_count();
    if (sms <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    TreeArgs a = {};
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.v_cache = static_cast<const __nv_bfloat16 *>(v_cache);
    a.q_stride = q_row_stride;
    a.bt = block_tables;
    a.ctx = context_lens;
    a.lens = draft_lens;
    a.mask = reinterpret_cast<const unsigned long long *>(tree_mask);
    a.max_blocks = max_blocks_per_seq;
    a.batch = batch;
    a.drafts = num_drafts;
    a.Hq = num_q_heads;
    a.Hkv = num_kv_heads;
    a.G = G;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    int r = TILE;
    while (block_size % r) r /= 2;
    a.box_rows = r;
    a.checked = checked_mode() ? 1 : 0;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.count = static_cast<int *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + l.parts);
    a.part_rows = l.part_rows;
    a.err = device_error_ptr();
    CUtensorMap tmk, tmv;
    const int64_t slots = (int64_t)num_blocks * block_size;
    pa_status st = encode_halves_map(&tmk, k_cache, slots, (int64_t)num_kv_heads * D * 2, num_kv_heads, r, r == TILE ? 2 : 1);
    if (st != PA_OK) return st;
    st = encode_halves_map(&tmv, v_cache, slots, (int64_t)num_kv_heads * D * 2, num_kv_heads, r, r == TILE ? 2 : 1);
    if (st != PA_OK) return st;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(std::min(sms, kMaxGrid), a_seq * batch / kMinTiles));
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    return l.nt == 1 ? launch_tree<1>(tmk, tmv, a, (int)grid, cs) : launch_tree<2>(tmk, tmv, a, (int)grid, cs);
}

}  // extern "C"
