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
//   warp 0     Q rows and K tiles by TMA, block ids 32 at a time
//   warp 1     S = Q K^T (M = 128, N = 64, K = 128) into one of a row tile's two TMEM
//              buffers
//   warp 2     O += P V (P from TMEM, V as an MN-major operand)
//   warp 3     V tiles by TMA
//   warps 4..  one thread per row: online softmax in base 2, P over S as bf16
// Of the 128 rows of an MMA only the live ones are loaded and read back; the
// others hold whatever the memory held, which cannot reach a live row.
//
// An item cut between CTAs leaves (m, l, o) of its parts in fp32 in the workspace, and
// the CTA in whose range it begins a note of it; a second kernel combines the parts, a
// CTA for 32 rows, in order.  (Combined by the CTA whose part came last, 256 rows of
// four parts took it 12 to 23 us, while the others were idle: 64 drafts over 8 x 32768
// keys 243 us instead of 229, over 4 x 2900 50 instead of 30.)  Short items are not cut.
//
// What bounds it: up to 128 rows per kv head the bytes of K and V (Qwen3-8B shape,
// 256 sequences x 4 drafts: 264 us, 6.6 TB/s); two row tiles the chain of products
// and softmax (64 drafts over 8 x 32768 keys: 230 us in a dozen calls, 252 in calls over
// some hundred milliseconds, 1.2 and 1.1 PFLOP/s, 70 and 64 % of the bytes' floor), in
// which a product's 64 keys re-read 128 rows of Q from shared memory.  Products of 128
// keys halve that but leave one score buffer a row tile: 34 us more.
//
// P is rounded to bf16, V's type, as the instruction takes both operands in one: an
// output is then off by 2.3e-3 of itself (root mean square, against 64 bits), 1.7e-3 by
// its own rounding.  l is summed from the rounded P that the product uses, so that the
// weights sum to one as they are.
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
constexpr uint32_t SBO = 1024;           // 8 rows x 128 B between core-matrix groups
constexpr uint32_t IDESC_S = idesc_bf16_f32(ROWS, TILE, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(ROWS, D, false, true);
constexpr int kMaxBatch = 2048;
constexpr int kMaxDrafts = 64;
constexpr int kMaxGrid = 256;
constexpr int kMinTiles = 2;             // a CTA's share at least
// What cutting items costs, in tiles: the parts' way through the workspace and the second
// kernel.  Items are left whole where that costs less.
__host__ __device__ constexpr int cut_tiles(bool pair) { return pair ? 10 : 6; }
constexpr float kLazy = 8.f;             // log2 headroom before the running maximum must move
constexpr unsigned FULL = 0xffffffffu;

// PAIR: an item has up to two row tiles, which share its K/V tiles.  Otherwise it
// has one, and consecutive items alternate between the two row-tile sets (Q,
// scores, O and softmax warps), so that one item's start and end run beside the
// other's tiles.
constexpr int THREADS = 384;
constexpr int KMAX = 6, VMAX = 8;                // ring stages at most
enum {  // barriers: rings, then per row tile [2] (and score buffer [2])
    KFULL = 0, KEMPTY = KFULL + KMAX, VFULL = KEMPTY + KMAX, VEMPTY = VFULL + VMAX, SFULL = VEMPTY + VMAX,
    PFULL = SFULL + 4, PDONE = PFULL + 4, OEMPTY = PDONE + 4, QFULL = OEMPTY + 2, QEMPTY = QFULL + 2,
    DRAIN = QEMPTY + 2, NBAR = DRAIN + 2
};
// Shared memory: Q [2], the rings, then from off_bar on the barriers, a few words
// (TMEM address, abort, mark, the longest item's tiles, scan scratch [12]), and per
// sequence the running sum of tiles, the length (int) and the drafts (byte).
constexpr int MISC = (NBAR * 8 + 15) / 16 * 16, ARRAYS = MISC + 128;
constexpr uint32_t TMEM_COLS = 512, COL_O = 256;               // S(h, b) at h * 128 + b * 64, O(h) at COL_O + h * 128
constexpr int kMaxSmem = 232448;
constexpr int fixed_smem(int batch) { return 1024 + ARRAYS + 9 * (batch + 1); }

// Floats of a part: o [D / 4][rows][4], so that the lanes of a warp, a row each, write and
// read whole lines, then (m, l) [rows]; a multiple of 32 bytes.
__host__ __device__ constexpr size_t slot_of(int rows) { return ((size_t)rows * (D + 2) + 7) / 8 * 8; }

// What CTA c leaves of the item that begins in its range and ends behind it: its output
// and rows, and the parts, the first in slot 2 c + 1, the others in 2 (c + i lanes).
struct TreeJob {
    int b, g, row0, rows, nparts, pad[3];  // nparts 0: none
};

struct TreeArgs {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *v_cache;
    const int32_t *bt, *ctx, *lens;
    const unsigned long long *mask;  // null: a chain
    int32_t max_blocks, batch, drafts, Hq, Hkv, G, block_size, num_blocks, box_rows, q_box, checked;
    int32_t q_rows;          // rows that a Q tile has room for (a multiple of 8): the MMA reads on past them
    int32_t k_stages, v_stages;
    int32_t shift;           // G = 1 << shift
    int32_t lanes;           // ranges side by side, each over Hkv / lanes of the heads
    int32_t whole;           // no item is cut
    float scale_log2;
    TreeJob *jobs;  // [grid]
    float *parts;  // [grid][2] of slot_of(part_rows)
    int32_t part_rows;
    DevError *err;
};

// A wait that is not over at once.  (A call of its own: inlined in the 25 places
// that wait, it takes the roles' loops apart in the instruction cache.)
__device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *abort, DevError *err, int where) {
    if (*abort) return false;
    if (mbar_wait(bar, parity)) return true;
    record_error(err, PA_DEV_TIMEOUT, where);
    *abort = 1;
    return false;
}
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort, DevError *err,
                                              int where) {
    if (__builtin_expect(mbar_try_wait(smem_addr(bar), parity), 1)) return true;
    return wait_on(bar, parity, abort, err, where);
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
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
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

// A part of an item that is a CTA's.
struct Seg {
    int b, g, blk;       // sequence, kv head, row block
    int t0, t1, nt;      // tiles [t0, t1) of nt
    int rows;            // live rows of the item
    uint32_t first;      // the item's first tile among the lane's
};

// Walks the segments of a CTA's range of tiles; every role of the CTA makes the
// same walk.
template <bool PAIR>
struct Walker {
    static constexpr int BLOCK = PAIR ? 2 * ROWS : ROWS;  // rows of an item
    const int *ctx_s;
    const uint8_t *n_s;
    const uint32_t *cum;
    int G, g0;  // the lane's first head
    uint32_t x, x1;
    int b;
    __device__ __forceinline__ int find(uint32_t at, int batch) const {
        int lo = 0, hi = batch - 1;  // the last b with cum[b] <= at
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cum[mid] <= at) lo = mid; else hi = mid - 1;
        }
        return lo;
    }
    // The first item's begin from `at` on.
    __device__ __forceinline__ uint32_t begin(uint32_t at, int batch) const {
        if (at >= cum[batch]) return cum[batch];
        const int i = find(at, batch);
        const uint32_t nt = (uint32_t)(ctx_s[i] + TILE - 1) / TILE;
        return cum[i] + (at - cum[i] + nt - 1) / nt * nt;
    }
    __device__ __forceinline__ void start(uint32_t x0, uint32_t xe, int batch, bool uncut) {
        x = uncut ? begin(x0, batch) : x0;
        x1 = uncut ? begin(xe, batch) : xe;
        b = find(x, batch);
    }
    // The next item in the range.
    __device__ __forceinline__ bool next(Seg &s) {
        if (x < x1) {
            while (cum[b + 1] <= x) ++b;
            const int nt = (ctx_s[b] + TILE - 1) / TILE, rows = n_s[b] * G;
            const int blocks = (rows + BLOCK - 1) / BLOCK;
            const uint32_t local = x - cum[b], it = local / (uint32_t)nt;
            const uint32_t first = cum[b] + it * (uint32_t)nt;
            s.b = b;
            s.g = g0 + (PAIR ? (int)it / blocks : (int)it);
            s.blk = PAIR ? (int)it % blocks : 0;
            s.t0 = (int)(x - first);
            x = min(first + (uint32_t)nt, x1);
            s.t1 = (int)(x - first);
            s.nt = nt;
            s.rows = min(rows - s.blk * BLOCK, BLOCK);
            s.first = first;
            return true;
        }
        return false;
    }
};

// Adds the V values of drafts lo .. hi - 1 that are not finite to a thread's row where its
// mask has them; element c of the row is at row[c / 4 * apart + c % 4] (fp32, or the bf16
// output).  Rare, and kept out of the loop's code.
__device__ __noinline__ void add_hidden(void *row, bool bf16, int apart, unsigned long long mask,
                                        const __nv_bfloat16 *v, int64_t v_row, const int32_t *bt, int block_size,
                                        int num_blocks, int first, int lo, int hi, int lane) {
    for (int j = lo; j < hi; ++j) {
        const int p = first + j, blk = __ldg(bt + p / block_size);
        if (blk < 0 || blk >= num_blocks) continue;
        const int64_t slot = (int64_t)blk * block_size + p % block_size;
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(v + slot * v_row) + lane);
        if (!__any_sync(FULL, not_finite2(w.x) || not_finite2(w.y))) continue;
        for (int c = 0; c < D; ++c) {
            const uint32_t t = __shfl_sync(FULL, (c & 2) ? w.y : w.x, c >> 2);
            const float x = (c & 1) ? bf16hi(t) : bf16lo(t);
            if (isfinite(x) || !((mask >> j) & 1)) continue;
            const int at = (c >> 2) * apart + (c & 3);
            if (bf16) {
                __nv_bfloat16 *e = static_cast<__nv_bfloat16 *>(row) + at;
                *e = __float2bfloat16(__bfloat162float(*e) + x);
            } else {
                static_cast<float *>(row)[at] += x;
            }
        }
    }
}

template <bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const __grid_constant__ TreeArgs a) {
    constexpr int BLOCK = Walker<PAIR>::BLOCK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int qhalf = a.q_rows * 128, qtile = 2 * qhalf;
    uint8_t *k_ring = smem + 2 * qtile, *v_ring = k_ring + a.k_stages * KV_BYTES;
    uint8_t *ctl = v_ring + a.v_stages * KV_BYTES;
    uint64_t *bar = reinterpret_cast<uint64_t *>(ctl);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ctl + MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(ctl + MISC + 4);
    uint32_t *wsum = reinterpret_cast<uint32_t *>(ctl + MISC + 48);
    uint32_t *cum = reinterpret_cast<uint32_t *>(ctl + ARRAYS);
    int *ctx_s = reinterpret_cast<int *>(cum + (a.batch + 1));
    uint8_t *n_s = reinterpret_cast<uint8_t *>(ctx_s + (a.batch + 1));
    const int warp = __shfl_sync(FULL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform, and known to be)

    static_assert(NBAR <= 64, "a thread of warps 2 and 3 each");
    if (threadIdx.x >= 64 && threadIdx.x < 64 + NBAR) {
        const int i = threadIdx.x - 64;
        // The four softmax warps of a row tile arrive one each.
        const bool per_warp = (i >= PFULL && i < PFULL + 4) || (i >= OEMPTY && i < OEMPTY + 2);
        mbar_init(&bar[i], per_warp ? 4u : 1u);
        fence_mbar_init();
    }
    if (threadIdx.x < 3) abort[threadIdx.x] = 0;  // and the words behind it
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    pdl_wait_then_release();
    if (threadIdx.x == 0) a.jobs[blockIdx.x].nparts = 0;
    // Lengths, and the running sum of the sequences' tiles.
    uint32_t carry = 0;
    int longest = 0;
    for (int base = 0; base < a.batch; base += THREADS) {
        const int b = base + threadIdx.x;
        uint32_t u = 0;
        if (b < a.batch) {
            int ctx = __ldg(a.ctx + b);
            int n = a.lens ? __ldg(a.lens + b) : ctx > 0 ? a.drafts : 0;
            if (ctx < 0 || ctx > (int64_t)a.max_blocks * a.block_size || n < 0 || n > a.drafts || n > ctx) {
                if (blockIdx.x == 0) record_error(a.err, PA_DEV_BAD_CONTEXT, b);
                n = 0;
            }
            if (n == 0) ctx = 0;
            ctx_s[b] = ctx;
            n_s[b] = (uint8_t)n;
            const int blocks = (n * a.G + BLOCK - 1) / BLOCK;
            longest = max(longest, (ctx + TILE - 1) / TILE);
            u = (uint32_t)((ctx + TILE - 1) / TILE) * (uint32_t)(a.Hkv / a.lanes * blocks);
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
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        if (b < a.batch) cum[b] = before + inc - u;
        carry = all;
        __syncthreads();
    }
    if (threadIdx.x == 0) cum[a.batch] = carry;
    longest = __reduce_max_sync(FULL, longest);
    if (lane == 0) atomicMax(const_cast<int *>(abort) + 2, longest);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The lane's tiles, its ranges, and this CTA's.  Items stay whole where that is shorter,
    // as if all were as long as the longest (16 sequences of 1000 keys, 8 heads of 4 x 64
    // rows: 31 us whole, 37 cut; 4 of 1900: 40 and 27): a range then goes from the first
    // item that begins in it to the first that begins behind it.
    const uint32_t P = carry, W0 = gridDim.x / (uint32_t)a.lanes, most = (uint32_t)abort[2];
    const uint64_t round = (uint64_t)most * W0;
    const uint32_t rounds = round >= P ? 1u : (P + (uint32_t)round - 1) / (uint32_t)round;
    const bool uncut = a.whole || rounds * most <= P / W0 + cut_tiles(PAIR);
    const uint32_t W = min(W0, max(1u, uncut ? P : P / kMinTiles));
    const uint32_t range = blockIdx.x / (uint32_t)a.lanes, side = blockIdx.x - range * (uint32_t)a.lanes;
    Walker<PAIR> walk{ctx_s, n_s, cum, a.G, (int)side * (a.Hkv / a.lanes), 0u, 0u, 0};
    if (range < W && P > 0)
        walk.start((uint32_t)((uint64_t)range * P / W), (uint32_t)((uint64_t)(range + 1) * P / W), a.batch, uncut);
    // Row tiles of segment number k.
    auto h_begin = [](int k) -> int { return PAIR ? 0 : k & 1; };
    auto h_end = [](int k, const Seg &s) -> int { return PAIR ? (s.rows + ROWS - 1) / ROWS : (k & 1) + 1; };
    // The MMA warps run whole and one lane issues: descriptors and addresses then stay
    // in uniform registers, where the instructions take them from.  (Issued by one lane
    // of a diverged warp they took 50 to 200 cycles each, and the issuing threads were
    // what bound the kernel: 64 drafts over 8 x 32768 keys 289 us instead of 252, the
    // Qwen3-8B shape 291 instead of 266.)
    uint32_t elected_;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(elected_));
    const bool elected = elected_ != 0;
    auto wwait = [&](int i, uint32_t parity, int where) -> bool {  // the warp as one
        return __all_sync(FULL, wait_or_abort(&bar[i], parity, abort, a.err, where));
    };
    Seg s;
    bool ok = true;

    // A ring's place: stage, and the parity of its current round.
    struct Ring {
        int n, st = 0;
        uint32_t par = 0;
        __device__ __forceinline__ Ring(int stages) : n(stages) {}
        __device__ __forceinline__ void next() {
            if (++st == n) {
                st = 0;
                par ^= 1u;
            }
        }
    };

    if (warp == 0 || warp == 3) {
        // ---------------------------------------------------------------- Q and K tiles; V tiles
        const bool is_k = warp == 0;
        const CUtensorMap *tm = is_k ? &tmk : &tmv;
        const int full = is_k ? KFULL : VFULL, empty = is_k ? KEMPTY : VEMPTY;
        uint8_t *base_tile = is_k ? k_ring : v_ring;
        Ring ring(is_k ? a.k_stages : a.v_stages);
        const int R = a.box_rows;
        uint32_t issued = 0, uq[2] = {0, 0};  // tiles, Q tiles
        // Block ids base + lane of a segment, the next one's fetched while this one is loaded.
        auto first_block = [&](const Seg &t) -> int { return t.t0 * TILE / a.block_size; };
        auto ids = [&](const Seg &t, int base) -> int {
            return __ldg(a.bt + (int64_t)t.b * a.max_blocks + min(base + lane, (ctx_s[t.b] - 1) / a.block_size));
        };
        Seg nx;
        bool have = walk.next(nx);
        int nid = have ? ids(nx, first_block(nx)) : 0;
        for (int k = 0; ok && have; ++k) {
            s = nx;
            int id = nid, base = first_block(s);
            have = walk.next(nx);
            if (have) nid = ids(nx, first_block(nx));
            const int key_end = ctx_s[s.b];
            if (is_k && lane == 0) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h < h_begin(k) || h >= h_end(k, s)) continue;
                    if (!(ok = wait_or_abort(&bar[QEMPTY + h], (uq[h] & 1u) ^ 1u, abort, a.err, 708))) break;
                    // Whole boxes, whatever the sequence's drafts: the rows past them are not live.
                    const int token = s.b * a.drafts + ((s.blk * BLOCK + (PAIR ? h * ROWS : 0)) >> a.shift);
                    mbar_arrive_expect_tx(&bar[QFULL + h], (uint32_t)(2 * a.q_box * a.G * 128));
                    tma_load_4d_plain(smem + h * qtile, &tmq, 0, s.g * a.G, token, 0, &bar[QFULL + h]);
                    tma_load_4d_plain(smem + h * qtile + qhalf, &tmq, 0, s.g * a.G, token, 1, &bar[QFULL + h]);
                    ++uq[h];
                }
            }
            for (int j = s.t0; j < s.t1; ++j) {
                const int nsub = (min(TILE, key_end - j * TILE) + R - 1) / R;
                if (lane == 0) {
                    ok = ok && wait_or_abort(&bar[empty + ring.st], ring.par ^ 1u, abort, a.err, is_k ? 700 : 701);
                    if (ok) mbar_arrive_expect_tx(&bar[full + ring.st], (uint32_t)(nsub * R * D * 2));
                }
                ok = __shfl_sync(FULL, ok ? 1 : 0, 0) != 0;
                if (!ok) break;
                for (int sub = 0; sub < nsub; ++sub) {
                    const int key = j * TILE + sub * R, lb = key / a.block_size;
                    if (lb >= base + 32) {
                        base = lb;
                        id = ids(s, base);
                    }
                    const int blk = __shfl_sync(FULL, id, lb - base);
                    if (lane == 0) {
                        const bool bad = blk < 0 || blk >= a.num_blocks;
                        if (bad && is_k && a.checked)
                            record_error(a.err, PA_DEV_BAD_BLOCK, (long long)s.b * a.max_blocks + lb);
                        // A box outside the pool is filled with zeros.
                        const int row = bad ? -2 * R : blk * a.block_size + key % a.block_size;
                        uint8_t *dst = base_tile + ring.st * KV_BYTES + sub * R * 128;
                        tma_load_4d_plain(dst, tm, 0, row, 0, s.g, &bar[full + ring.st]);
                        if (R != TILE) tma_load_4d_plain(dst + KV_HALF, tm, 0, row, 1, s.g, &bar[full + ring.st]);
                    }
                }
                ring.next();
                ++issued;
            }
        }
        if (lane == 0 && *abort) {  // issued copies land before the shared memory is given back
            for (uint32_t x = issued >= (uint32_t)ring.n ? issued - ring.n : 0; x < issued; ++x)
                (void)mbar_wait(&bar[full + x % ring.n], (x / ring.n) & 1u);
            for (int h = 0; h < 2; ++h)
                if (uq[h] > 0) (void)mbar_wait(&bar[QFULL + h], (uq[h] - 1) & 1u);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- S = Q K^T
        Ring ring(a.k_stages);
        uint32_t th[2] = {0, 0}, uq[2] = {0, 0};  // of each row tile: tiles, segments
        bool issued = false;
        for (int k = 0; ok && walk.next(s); ++k) {
            const int h0 = h_begin(k), h1 = h_end(k, s);
            for (int j = s.t0; ok && j < s.t1; ++j) {
                if (!(ok = wwait(KFULL + ring.st, ring.par, 703))) break;
                const uint64_t kdesc = smem_desc_sw128(smem_addr(k_ring + ring.st * KV_BYTES), 16, SBO);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h < h0 || h >= h1) continue;
                    const int b = th[h] & 1;
                    if (j == s.t0) {
                        if (!(ok = wwait(QFULL + h, uq[h] & 1u, 702))) break;
                        ++uq[h];
                    }
                    // The buffer is free once the P.V of two tiles ago has read it.
                    if (!(ok = wwait(PDONE + 2 * h + b, ((th[h] >> 1) & 1u) ^ 1u, 704))) break;
                    tc_fence_after();
                    const uint64_t qdesc = smem_desc_sw128(smem_addr(smem + h * qtile), 16, SBO);
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_bf16_ss(tmem + h * 128 + b * TILE,
                                        qdesc + (uint64_t)(((kk >> 2) * qhalf + (kk & 3) * 32) >> 4),
                                        kdesc + (uint64_t)(((kk >> 2) * KV_HALF + (kk & 3) * 32) >> 4), IDESC_S,
                                        kk > 0 ? 1u : 0u);
                        mma_commit(&bar[SFULL + 2 * h + b]);
                        if (j == s.t1 - 1) mma_commit(&bar[QEMPTY + h]);  // the segment's products have read Q
                    }
                    issued = true;
                    ++th[h];
                }
                if (!ok) break;
                if (elected) mma_commit(&bar[KEMPTY + ring.st]);
                ring.next();
            }
        }
        if (issued && elected && *abort) {
            mma_commit(&bar[DRAIN]);
            (void)mbar_wait(&bar[DRAIN], 0);
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- O += P V
        Ring ring(a.v_stages);
        uint32_t th[2] = {0, 0}, uh[2] = {0, 0};
        bool issued = false;
        for (int k = 0; ok && walk.next(s); ++k) {
            const int h0 = h_begin(k), h1 = h_end(k, s);
            for (int j = s.t0; ok && j < s.t1; ++j) {
                if (!(ok = wwait(VFULL + ring.st, ring.par, 705))) break;
                const int steps = (min(TILE, ctx_s[s.b] - j * TILE) + 15) / 16;  // keys past the last: P is 0
                const uint64_t vdesc = smem_desc_sw128(smem_addr(v_ring + ring.st * KV_BYTES), KV_HALF, SBO);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h < h0 || h >= h1) continue;
                    const int b = th[h] & 1;
                    if (j == s.t0) {  // O is free once the row tile's last segment was read
                        if (!(ok = wwait(OEMPTY + h, (uh[h] & 1u) ^ 1u, 706))) break;
                        ++uh[h];
                    }
                    if (!(ok = wwait(PFULL + 2 * h + b, (th[h] >> 1) & 1u, 707))) break;
                    tc_fence_after();
                    if (elected) {
                        // 16 keys a step = 8 TMEM columns of P; unrolled where it can be.
                        if (steps == TILE / 16) {
#pragma unroll
                            for (int kk = 0; kk < TILE / 16; ++kk)
                                mma_bf16_ts(tmem + COL_O + h * 128, tmem + h * 128 + b * TILE + kk * 8,
                                            vdesc + (uint64_t)((kk * 16 * 128) >> 4), IDESC_PV,
                                            (j > s.t0 || kk > 0) ? 1u : 0u);
                        } else {
#pragma unroll 1
                            for (int kk = 0; kk < steps; ++kk)
                                mma_bf16_ts(tmem + COL_O + h * 128, tmem + h * 128 + b * TILE + kk * 8,
                                            vdesc + (uint64_t)((kk * 16 * 128) >> 4), IDESC_PV,
                                            (j > s.t0 || kk > 0) ? 1u : 0u);
                        }
                        mma_commit(&bar[PDONE + 2 * h + b]);
                    }
                    issued = true;
                    ++th[h];
                }
                if (!ok) break;
                if (elected) mma_commit(&bar[VEMPTY + ring.st]);
                ring.next();
            }
        }
        if (issued && elected && *abort) {
            mma_commit(&bar[DRAIN + 1]);
            (void)mbar_wait(&bar[DRAIN + 1], 0);
        }
    } else {
        // ---------------------------------------------------------------- softmax, output
        const int h = (warp - 4) >> 2;  // row tile
        const int quarter = warp & 3;
        const int wrow = quarter * 32, row = wrow + lane;  // row of the tile == TMEM lane
        const uint32_t t_s = tmem + ((uint32_t)wrow << 16) + h * 128, t_o = tmem + ((uint32_t)wrow << 16) + COL_O + h * 128;
        const float sl = a.scale_log2;
        {
            // Tokens past a sequence's drafts: zeros.
            const int per = a.Hq * (D / 8);  // 16-byte chunks of a token
            for (int t = warp - 4 + 8 * blockIdx.x; t < a.batch * a.drafts; t += 8 * gridDim.x) {
                const int b = t / a.drafts;
                if (t - b * a.drafts < n_s[b]) continue;
                uint4 *dst = reinterpret_cast<uint4 *>(a.out) + (int64_t)t * per;
                for (int c = lane; c < per; c += 32) dst[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        // Set once a draft's V held something not finite, and never taken back: from then
        // on each segment looks for such values of its own.  (A mark per segment would need
        // a place that no warp writes again before the slowest has read it, and a warp
        // without live rows runs segments ahead of one that still stores its own.)
        volatile int *mark = abort + 1;
        // The next segment that this row tile has rows in: its first tile's number, and
        // (asked for ahead) this row's mask.
        int k_next = 0;
        uint32_t g_next = 0;
        struct Own {
            Seg s;
            uint32_t g;
            unsigned long long m;
        };
        auto fetch = [&](Own &o) -> bool {
            while (walk.next(o.s)) {
                const int k = k_next++;
                const uint32_t g = g_next;
                g_next += o.s.t1 - o.s.t0;
                if (h < h_begin(k) || h >= h_end(k, o.s)) continue;
                o.g = g;
                o.m = 0;
                const int row0 = PAIR ? h * ROWS : 0;
                if (row0 + row < o.s.rows) {
                    const int di = (o.s.blk * BLOCK + row0 + row) >> a.shift;
                    o.m = a.mask ? __ldg(a.mask + (int64_t)o.s.b * a.drafts + di) : di >= 63 ? ~0ull : (2ull << di) - 1;
                }
                return true;
            }
            return false;
        };
        Own nx;
        bool have = fetch(nx);
        uint32_t th = 0;  // tiles of this row tile
        while (ok && have) {
            s = nx.s;
            uint32_t gg = nx.g;
            unsigned long long m64 = nx.m;
            have = fetch(nx);
            const int row0 = PAIR ? h * ROWS : 0;
            const int live = min(s.rows - row0, ROWS);  // live rows of this row tile
            const int ctx = ctx_s[s.b], n = n_s[s.b], first = ctx - n;
            const bool mine = row < live, wlive = wrow < live;
            if (n < 64) m64 &= (1ull << n) - 1;
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = s.t0; ok && j < s.t1; ++j, ++gg, ++th) {
                const int b = th & 1, kb = j * TILE;
                const uint32_t cs = t_s + b * TILE;
                if (!(ok = wwait(SFULL + 2 * h + b, (th >> 1) & 1u, 710))) break;
                if (kb + TILE > first) {
                    // (V's place in its ring is waited for after the scores: their product
                    // followed the P.V of at most four tiles before, so that this tile's
                    // round is the next to complete, as a wait by parity needs.)
                    // A tile with drafts: V's rows past the last key that the
                    // product reads become zeros, and drafts' values that are not
                    // finite too.  Each row tile of the item does it before its
                    // product; what the first has mended, the second leaves.
                    const uint32_t round = gg / (uint32_t)a.v_stages, st = gg - round * (uint32_t)a.v_stages;
                    if (!(ok = wwait(VFULL + st, round & 1u, 709))) break;
                    const int kend = min(TILE, ctx - kb), kpad = (kend + 15) & ~15, k0 = max(0, first - kb);
                    const uint32_t vb = smem_addr(v_ring + st * KV_BYTES);
                    for (int i = threadIdx.x & 127; i < (kpad - k0) * 16; i += 128) {
                        const int r = k0 + (i >> 4), c = i & 15;
                        const uint32_t at = vb + (uint32_t)((c >> 3) * KV_HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                        const uint4 w = ld_shared_v4(at);
                        if (r >= kend) {
                            if (w.x | w.y | w.z | w.w) st_shared_u4(at, make_uint4(0u, 0u, 0u, 0u));
                        } else if (not_finite2(w.x) || not_finite2(w.y) || not_finite2(w.z) || not_finite2(w.w)) {
                            // Seen by every warp at the segment's end: its P follows this.
                            *mark = 1;
                            __threadfence_block();
                            st_shared_u4(at, make_uint4(finite_only(w.x), finite_only(w.y), finite_only(w.z),
                                                        finite_only(w.w)));
                        }
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_after();
                if (wlive) {
                    uint32_t r[TILE];
                    tmem_ld32(cs, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
                    tmem_ld32(cs + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
                    tmem_ld_wait();
                    if (kb + TILE > first) {
                        const int d = first - kb;  // keys of the tile before the drafts
                        unsigned long long vis;
                        if (d > 0) vis = ((1ull << d) - 1) | (m64 << d);
                        else vis = -d < 64 ? m64 >> -d : 0ull;
                        const uint32_t vlo = (uint32_t)vis, vhi = (uint32_t)(vis >> 32);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (!((vlo >> e) & 1u)) r[e] = __float_as_uint(-INFINITY);
                            if (!((vhi >> e) & 1u)) r[e + 32] = __float_as_uint(-INFINITY);
                        }
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < TILE / 2; ++e)
                        m4[e & 3] = max3(m4[e & 3], __uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    const bool grow_m = mine && (mx - m_run) * sl > kLazy;  // rows that are not live stay put
                    const float m_new = grow_m ? mx : m_run;
                    const float alpha = grow_m ? fast_exp2((m_run - m_new) * sl) : 1.f;
                    if (j > s.t0 && __any_sync(FULL, grow_m)) {
                        // O holds the products up to the previous tile before it is rescaled.
                        if (!(ok = wwait(PDONE + 2 * h + ((th - 1) & 1), ((th - 1) >> 1) & 1u, 711))) break;
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
                    float2 rs[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
                    const float2 sl2 = make_float2(sl, sl), nm2 = make_float2(neg_m, neg_m);
                    uint32_t pk[TILE / 2];
#pragma unroll
                    for (int e = 0; e < TILE / 2; ++e) {
                        const float2 x = fma2(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), sl2, nm2);
                        pk[e] = pack_bf16(fast_exp2(x.x), fast_exp2(x.y));
                        rs[e & 3] = add2(rs[e & 3], make_float2(bf16lo(pk[e]), bf16hi(pk[e])));
                    }
                    tmem_st32(cs, pk);  // P over the first 32 columns of the buffer
                    tmem_st_wait();
                    l_run += ((rs[0].x + rs[0].y) + (rs[1].x + rs[1].y)) + ((rs[2].x + rs[2].y) + (rs[3].x + rs[3].y));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[PFULL + 2 * h + b]);
            }
            if (!ok) break;
            // ---- the segment's rows
            if (!(ok = wwait(PDONE + 2 * h + ((th - 1) & 1), ((th - 1) >> 1) & 1u, 712))) break;
            tc_fence_after();
            const bool whole = s.t0 == 0 && s.t1 == s.nt;
            // A part: slot 1 of the item's first CTA, slot 0 of the others.
            int c0 = 0, nparts = 0;
            float *slot = nullptr;
            if (!whole) {  // the range that holds tile x: ((x + 1) W - 1) / P
                const int r0 = (int)(((uint64_t)(s.first + 1) * W - 1) / P);
                nparts = (int)(((uint64_t)(s.first + s.nt) * W - 1) / P) - r0 + 1;
                c0 = r0 * a.lanes + (int)side;
                slot = a.parts + (size_t)(2 * blockIdx.x + (blockIdx.x == c0 ? 1 : 0)) * slot_of(a.part_rows);
            }
            if (wlive) {
                const float inv = !whole ? 1.f : l_run == 0.f ? 0.f : 1.f / l_run;  // a row that sees nothing: zeros
                const int gr = s.blk * BLOCK + row0 + row;  // row of the (sequence, kv head)
                __nv_bfloat16 *dst =
                    a.out + (((int64_t)s.b * a.drafts + (gr >> a.shift)) * a.Hq + s.g * a.G + (gr & (a.G - 1))) * D;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tmem_ld32(t_o + c * 32, o);
                    tmem_ld_wait();
                    if (mine && whole) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t *v = &o[8 * e];
                            reinterpret_cast<uint4 *>(dst)[4 * c + e] =
                                make_uint4(pack_bf16(__uint_as_float(v[0]) * inv, __uint_as_float(v[1]) * inv),
                                           pack_bf16(__uint_as_float(v[2]) * inv, __uint_as_float(v[3]) * inv),
                                           pack_bf16(__uint_as_float(v[4]) * inv, __uint_as_float(v[5]) * inv),
                                           pack_bf16(__uint_as_float(v[6]) * inv, __uint_as_float(v[7]) * inv));
                        }
                    } else if (mine) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)  // a warp's stores: 512 bytes in a row
                            reinterpret_cast<uint4 *>(slot)[(size_t)(8 * c + e) * a.part_rows + row0 + row] =
                                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[OEMPTY + h]);
            if (wlive && __any_sync(FULL, *mark != 0)) {  // (the lanes as one: another warp may set it now)
                // What was taken out of V: added to the rows that see it.
                const int lo = max(0, s.t0 * TILE - first), hi = min(n, s.t1 * TILE - first);  // drafts of the segment
                const int gr = s.blk * BLOCK + row0 + row;
                const int64_t head = ((int64_t)s.b * a.drafts + (gr >> a.shift)) * a.Hq + s.g * a.G + (gr & (a.G - 1));
                void *at = whole ? static_cast<void *>(a.out + head * D)
                                 : static_cast<void *>(slot + (size_t)(row0 + row) * 4);
                add_hidden(at, whole, whole ? 4 : a.part_rows * 4, mine ? m64 : 0ull, a.v_cache + (int64_t)s.g * D,
                           (int64_t)a.Hkv * D, a.bt + (int64_t)s.b * a.max_blocks, a.block_size, a.num_blocks, first, lo,
                           hi, lane);
            }
            if (whole) continue;
            if (mine) reinterpret_cast<float2 *>(slot + (size_t)a.part_rows * D)[row0 + row] = make_float2(m_run * sl, l_run);
            if (quarter == 0 && lane == 0 && blockIdx.x == c0 && (!PAIR || h == 0))
                a.jobs[c0] = {s.b, s.g, s.blk * BLOCK, s.rows, nparts, {}};
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
}

// Combines the parts of the items that were cut: a CTA for 32 rows (blockIdx.y) of the item
// of blockIdx.x and D / Z of its columns; a warp 16 columns of every Z-th part, four parts
// under way.  A part's m of -inf has seen nothing; NaN in l or o goes on.
struct CombineArgs {
    __nv_bfloat16 *out;
    const TreeJob *jobs;
    const float *parts;
    int part_rows, lanes, drafts, Hq, G, shift;
};
struct Sums {
    float m = -INFINITY, l = 0.f;
    float4 o[4] = {};
    // Scales to a maximum of mn; returns what -inf counts as.
    __device__ __forceinline__ float raise(float mn) {
        const float ref = mn == -INFINITY ? 0.f : mn, f = fast_exp2(m - ref);
        m = mn;
        l *= f;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = make_float4(o[e].x * f, o[e].y * f, o[e].z * f, o[e].w * f);
        return ref;
    }
    __device__ __forceinline__ void add(float mp, float lp, const float4 (&v)[4], float ref) {
        const float f = fast_exp2(mp - ref);
        l = fmaf(lp, f, l);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = make_float4(fmaf(v[e].x, f, o[e].x), fmaf(v[e].y, f, o[e].y), fmaf(v[e].z, f, o[e].z),
                               fmaf(v[e].w, f, o[e].w));
    }
};
constexpr int CTHREADS = 256;
template <int Z>
__global__ void __launch_bounds__(CTHREADS) combine_kernel(const __grid_constant__ CombineArgs a) {
    pdl_wait_then_release();
    constexpr int SETS = 8 / Z, PM = 4;  // sets of 16 columns; parts at a time
    const int4 job = __ldcg(reinterpret_cast<const int4 *>(a.jobs + blockIdx.x));
    const int nparts = __ldcg(&a.jobs[blockIdx.x].nparts);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y * 32 + lane;
    if (nparts == 0 || (int)blockIdx.y * 32 >= job.w) return;
    const int set = warp % SETS + blockIdx.z * SETS, p0 = warp / SETS;
    const bool mine = row < job.w;
    const size_t slot = slot_of(a.part_rows);
    const float *rest = a.parts + (size_t)2 * blockIdx.x * slot;
    Sums sum;
#pragma unroll 1
    for (int i0 = p0; i0 < nparts; i0 += PM * Z) {
        float4 v[PM][4];
        float2 ml[PM];
        float mn = sum.m;
#pragma unroll
        for (int p = 0; p < PM; ++p) {
            const int i = i0 + p * Z;
            ml[p] = make_float2(-INFINITY, 0.f);
            if (i < nparts && mine) {
                const float *from = i == 0 ? rest + slot : rest + (size_t)(2 * i * a.lanes) * slot;
                ml[p] = __ldcg(reinterpret_cast<const float2 *>(from + (size_t)a.part_rows * D) + row);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[p][e] = __ldcg(reinterpret_cast<const float4 *>(from) + (size_t)(4 * set + e) * a.part_rows + row);
            }
        }
#pragma unroll
        for (int p = 0; p < PM; ++p) mn = fmaxf(mn, ml[p].x);
        const float ref = sum.raise(mn);
#pragma unroll
        for (int p = 0; p < PM; ++p)
            if (i0 + p * Z < nparts) sum.add(ml[p].x, ml[p].y, v[p], ref);
    }
    if (Z > 1) {
        __shared__ float4 os[8][4][32];
        __shared__ float2 mls[8][32];
        if (p0 > 0) {
            mls[warp][lane] = make_float2(sum.m, sum.l);
#pragma unroll
            for (int e = 0; e < 4; ++e) os[warp][e][lane] = sum.o[e];
        }
        __syncthreads();
        if (p0 > 0) return;
#pragma unroll 1
        for (int w = warp + SETS; w < 8 && w / SETS < nparts; w += SETS) {
            const float2 ml = mls[w][lane];
            float4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = os[w][e][lane];
            const float ref = sum.raise(fmaxf(sum.m, ml.x));
            sum.add(ml.x, ml.y, v, ref);
        }
    }
    if (!mine) return;
    const float inv = sum.l == 0.f ? 0.f : 1.f / sum.l;
    const int gr = job.z + row;
    uint4 *dst = reinterpret_cast<uint4 *>(
        a.out + (((int64_t)job.x * a.drafts + (gr >> a.shift)) * a.Hq + job.y * a.G + (gr & (a.G - 1))) * D + 16 * set);
#pragma unroll
    for (int e = 0; e < 4; e += 2)
        dst[e / 2] = make_uint4(pack_bf16(sum.o[e].x * inv, sum.o[e].y * inv), pack_bf16(sum.o[e].z * inv, sum.o[e].w * inv),
                                pack_bf16(sum.o[e + 1].x * inv, sum.o[e + 1].y * inv),
                                pack_bf16(sum.o[e + 1].z * inv, sum.o[e + 1].w * inv));
}

// Notes of the items that were cut, then the parts.
struct Layout {
    bool pair;
    int part_rows;  // rows of an item at most
    size_t parts, bytes;
};
Layout layout_of(int drafts, int G) {
    Layout l;
    l.pair = drafts * G > ROWS;
    l.part_rows = std::min(drafts * G, 2 * ROWS);
    l.parts = (size_t)kMaxGrid * sizeof(TreeJob);
    l.bytes = l.parts + (size_t)kMaxGrid * 2 * slot_of(l.part_rows) * sizeof(float);
    return l;
}

// Per (device, variant): the shared-memory attribute has been set.
std::atomic<int> g_attr_done[64][2];

template <bool PAIR>
pa_status launch_tree(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv, const TreeArgs &a,
                      int grid, bool is_short, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= 64) return fail(PA_ERR_UNSUPPORTED, "device %d", dev);
    if (!g_attr_done[dev][PAIR].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(decode_tree_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxSmem);
        if (e != cudaSuccess) return cuda_fail(e, "decode_tree_kernel shared memory");
        g_attr_done[dev][PAIR].store(1, std::memory_order_release);
    }
    const size_t smem = (size_t)4 * a.q_rows * 128 + (size_t)(a.k_stages + a.v_stages) * KV_BYTES + fixed_smem(a.batch);
    // The set-up beside the end of the kernel before: after a pa_rope_store_kvcache on a
    // stream, Qwen3-0.6B shape with 8 drafts 94.8 us for both, 96.8 with a plain launch; 1 x
    // 1000 keys 10.6 and 11.1.  But the CTAs then take the SMs in the order in which the
    // kernel before leaves them, and those of a range need not sit side by side, which
    // long calls feel (Qwen3-8B shape in a graph 273.3 us for both, 271.8 so): they have a
    // plain launch.
    if (is_short)
        return launch_pdl(decode_tree_kernel<PAIR>, dim3((unsigned)grid), dim3(THREADS), smem, stream,
                          "decode_tree_kernel", tmq, tmk, tmv, a);
    decode_tree_kernel<PAIR><<<dim3((unsigned)grid), dim3(THREADS), smem, stream>>>(tmq, tmk, tmv, a);
    return check_launch("decode_tree_kernel");
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
    const int64_t blocks = (num_drafts * G + 2 * ROWS - 1) / (2 * ROWS);
    const int64_t a_seq = (int64_t)num_kv_heads * blocks * ((keys + TILE - 1) / TILE);
    if (num_kv_heads > (1 << 16) || a_seq > 0x7fffffffLL / batch)
        return fail(PA_ERR_UNSUPPORTED, "too many tiles (batch * num_kv_heads * max_blocks_per_seq * block_size)");
    if (!workspace || workspace_bytes < l.bytes)
        return fail(PA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : (size_t)0, l.bytes);
    if (reinterpret_cast<uintptr_t>(workspace) & 31u) return fail(PA_ERR_INVALID_ARG, "workspace must be 32-byte aligned");
    const int sms = sm_count();
    if (sms <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    TreeArgs a = {};
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.v_cache = static_cast<const __nv_bfloat16 *>(v_cache);
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
    while ((1 << a.shift) < G) ++a.shift;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    int r = TILE;
    while (block_size % r) r /= 2;
    a.box_rows = r;
    a.checked = checked_mode() ? 1 : 0;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.jobs = static_cast<TreeJob *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + l.parts);
    a.part_rows = l.part_rows;
    a.err = device_error_ptr();
    a.q_box = std::min(num_drafts, ROWS / G);
    // Few rows leave room for more K and V in flight.  A V tile is held until its
    // P.V is done, a K tile only until its scores are: V gets the larger share.
    a.q_rows = std::min(ROWS, (a.q_box * G + 7) / 8 * 8);
    const int tiles = std::min(KMAX + VMAX, (kMaxSmem - fixed_smem(batch) - 4 * a.q_rows * 128) / KV_BYTES);
    a.k_stages = std::min(KMAX, tiles * 3 / 7);
    a.v_stages = std::min(VMAX, tiles - a.k_stages);
    CUtensorMap tmq, tmk, tmv;
    pa_status st = encode_token_heads_map(&tmq, q, (int64_t)batch * num_drafts, q_row_stride * 2, num_q_heads, G, a.q_box);
    if (st != PA_OK) return st;
    const int64_t slots = (int64_t)num_blocks * block_size;
    st = encode_halves_map(&tmk, k_cache, slots, (int64_t)num_kv_heads * D * 2, num_kv_heads, r, r == TILE ? 2 : 1);
    if (st != PA_OK) return st;
    st = encode_halves_map(&tmv, v_cache, slots, (int64_t)num_kv_heads * D * 2, num_kv_heads, r, r == TILE ? 2 : 1);
    if (st != PA_OK) return st;
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(std::min(sms, kMaxGrid), a_seq * batch / kMinTiles));
    // Side by side, the CTAs of a range walk the same keys of different heads at
    // the same time, so that the pool's rows (all heads of a token) are read whole.
    // As many lanes as leave at most a tenth of the CTAs without work.
    a.lanes = 1;
    for (int n = 2; n <= num_kv_heads && n <= grid; ++n)
        if (num_kv_heads % n == 0 && grid / n * n * 10 >= grid * 9) a.lanes = n;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    // Tables too short for a cut: one launch.  So too two tiles more, which is what the second
    // launch costs, where every item has a CTA of its own (whatever the lengths: the
    // table's width may be one sequence's alone).  Device us, one launch and two, the second
    // of which combines nothing up to here: 1 and 4 sequences, 8 kv heads, 5 drafts, 512 keys
    // 10.4 and 11.4, 10.9 and 12.0; 64 drafts, 768 keys 19.9 and 21.5.  A tile more, which
    // is cut: 5 drafts, 576 keys 11.1 and 10.0, 11.6 and 11.5; 64 drafts, 832 keys 20.9 and
    // 15.2, 21.3 and 23.2.
    const int64_t longest = (keys + TILE - 1) / TILE;
    a.whole = longest <= cut_tiles(l.pair) ||
              (longest <= cut_tiles(l.pair) + 2 && (int64_t)batch * num_kv_heads * blocks <= grid);
    const bool is_short = a_seq * batch <= 512 * grid;  // tiles a CTA at most
    st = l.pair ? launch_tree<true>(tmq, tmk, tmv, a, (int)grid, is_short, cs)
                : launch_tree<false>(tmq, tmk, tmv, a, (int)grid, is_short, cs);
    if (st != PA_OK || a.whole) return st;
    const CombineArgs c = {a.out, a.jobs, a.parts, a.part_rows, a.lanes, a.drafts, a.Hq, a.G, a.shift};
    // Many parts an item: its columns over more CTAs, and the parts over more warps.  (CTAs
    // without work cost too: Qwen3-0.6B shape, 8 drafts, 84.6 us with one CTA a note, 89.8
    // with 8.)
    const int64_t rows32 = (l.part_rows + 31) / 32, parts = grid / (num_kv_heads * blocks * batch);
    const int z = l.pair || parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : 8;
    const auto kernel = z == 8   ? combine_kernel<8>
                        : z == 4 ? combine_kernel<4>
                        : z == 2 ? combine_kernel<2>
                                 : combine_kernel<1>;
    return launch_pdl(kernel, dim3((unsigned)grid, (unsigned)rows32, z), dim3(CTHREADS), 0, cs, "combine_kernel", c);
}

}  // extern "C"
