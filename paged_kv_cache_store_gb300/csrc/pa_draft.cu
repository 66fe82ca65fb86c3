// pa_draft.cu -- what surrounds the attention of a tree of drafted tokens: its
// masks, positions and slots, the verification of the drafts, and the move of
// the kept rows next to the context.
//
// Verification, per sequence: node 0 is the token that the drafts continue, node
// i > 0 a drafted token under parent[i] < i.  At a node v with target
// probabilities p = softmax(logits_v / T), w = p and s = 1, for its children in
// order, child c with token x and given number u:
//   kept if u q(x) s < w(x),  else w <- max(w - s q, 0), s <- sum w,
// q = draft_probs_v, the distribution that the children were drawn from, each on
// its own.  (u < ratio of the normalised w / s to q, without a division.)  Unrolled,
// w = max(p - S q, 0) with S the sum of the s so far: a scalar carries the whole
// state, and w is never written.  Without draft_probs the children are chosen
// candidates, q is 1 at the child's token: w(x) <- 0.  The walk goes on from a
// kept child; where none is kept, the last token is argmax w / max(E, 1e-10), E the
// given exponential numbers: a draw from w / s.
//
// How: a thread-block cluster per sequence walks its tree, so only the rows of
// the nodes that are reached are read.  A node costs one pass over its logits
// (maximum and sum), one more per rejected child that has a sibling after it, and
// the last node one pass for the draw (its logits from L2).  What bounds it is the
// latency of that chain of passes, a cluster barrier each: 32 trees of 32 nodes and 151936
// bf16 logits take 33 to 41 us by their paths, 6 us of them the bytes of the rows reached
// at the copy's rate.  Small rows and short chains are therefore read all at once, ahead
// of the walk (kAtOnceBytes): 64 drawn chains of 6 nodes take 49 us for 190 MB, of which
// the rows reached are 23 us; no pipe is full (HBM 46 %, issue slots 45 %, exponentials 22
// %), the loads under way, 32 KiB an SM, are fewer than HBM's latency asks for.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kMaxNodes = 64;

// ---------------------------------------------------------------------------
// Masks, positions and slots
// ---------------------------------------------------------------------------
struct MetaArgs {
    unsigned long long *mask;
    int32_t *positions, *slots;
    const int32_t *parents, *ctx, *lens, *bt;
    int32_t max_blocks, batch, nodes, block_size;
    DevError *err;
};

// Tree size of sequence b: draft_lens, or all nodes of a row with a context; 0
// (recorded) where the lengths do not fit.
__device__ __forceinline__ int tree_size(int ctx, const int32_t *lens, int b, int nodes, int64_t limit, bool &bad) {
    const int n = lens ? __ldg(lens + b) : (ctx > 0 ? nodes : 0);
    bad = ctx < 0 || ctx > limit || n < 0 || n > nodes || n > ctx;
    return bad ? 0 : n;
}

// A thread per node walks up to the root.
__global__ void __launch_bounds__(128) tree_metadata_kernel(const __grid_constant__ MetaArgs a) {
    pdl_wait_then_release();
    const int64_t t = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (t >= (int64_t)a.batch * a.nodes) return;
    const int b = (int)(t / a.nodes), i = (int)(t - (int64_t)b * a.nodes);
    const int ctx = __ldg(a.ctx + b);
    bool bad;
    const int n = tree_size(ctx, a.lens, b, a.nodes, (int64_t)a.max_blocks * a.block_size, bad);
    if (bad && i == 0) record_error(a.err, PA_DEV_BAD_CONTEXT, b);
    if (i >= n) {
        a.mask[t] = 0;
        a.positions[t] = 0;
        a.slots[t] = -1;
        return;
    }
    unsigned long long m = 1ull << i;
    int v = i, depth = 0;
    while (v > 0) {
        const int p = a.parents ? __ldg(a.parents + (int64_t)b * a.nodes + v) : v - 1;
        if (p < 0 || p >= v) {
            if (v == i) record_error(a.err, PA_DEV_BAD_TREE, t);
            break;
        }
        m |= 1ull << p;
        ++depth;
        v = p;
    }
    a.mask[t] = m;
    a.positions[t] = ctx - n + depth;
    const int p = ctx - n + i, blk = __ldg(a.bt + (int64_t)b * a.max_blocks + p / a.block_size);
    const int64_t slot = (int64_t)blk * a.block_size + p % a.block_size;
    if (slot > INT32_MAX) record_error(a.err, PA_DEV_BAD_BLOCK, (long long)b * a.max_blocks + p / a.block_size);
    a.slots[t] = slot < 0 || slot > INT32_MAX ? -1 : (int32_t)slot;
}

// ---------------------------------------------------------------------------
// Moving the kept rows
// ---------------------------------------------------------------------------
constexpr int MOVE_THREADS = 256;

struct MoveArgs {
    uint4 *k, *v;
    int64_t k_layer, v_layer;  // 16-byte units between layers
    const int32_t *bt, *ctx, *lens, *nodes, *counts;
    int32_t max_blocks, batch, width, layers, row16, block_size, num_blocks;
    DevError *err;
};

// A CTA takes a sequence and a share of its (layer, K or V, 16-byte column)
// items.  nodes[j] >= j along a path, so a row is never written before it is read
// as long as a column's rows are moved in order; up to eight loads are in flight.
__global__ void __launch_bounds__(MOVE_THREADS) compact_kernel(const __grid_constant__ MoveArgs a) {
    pdl_wait_then_release();
    __shared__ int64_t src[kMaxNodes], dst[kMaxNodes];
    __shared__ int moves;
    const int b = blockIdx.x, lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        const int ctx = __ldg(a.ctx + b);
        bool bad;
        const int n = tree_size(ctx, a.lens, b, a.width, (int64_t)a.max_blocks * a.block_size, bad);
        if (bad && lane == 0 && blockIdx.y == 0) record_error(a.err, PA_DEV_BAD_CONTEXT, b);
        const int count = min(max(__ldg(a.counts + b), 0), n), base = ctx - n;
        const int32_t *bt = a.bt + (int64_t)b * a.max_blocks;
        int total = 0;
        bool stop = false;
        for (int j0 = 0; j0 < count; j0 += 32) {
            const int j = j0 + lane;
            int node = j;
            bool wrong = false;
            if (j < count) {
                node = __ldg(a.nodes + (int64_t)b * a.width + j);
                const int prev = j ? __ldg(a.nodes + (int64_t)b * a.width + j - 1) : -1;
                wrong = node <= prev || node >= n || (j == 0 && node != 0);
            }
            const unsigned w = __ballot_sync(FULL, wrong);
            if (w && lane == 0 && blockIdx.y == 0)
                record_error(a.err, PA_DEV_BAD_TREE, (long long)b * a.width + j0 + __ffs(w) - 1);
            const bool before = !stop && (w == 0 || j < j0 + __ffs(w) - 1);  // the path up to its first bad node
            stop = stop || w != 0;
            bool go = before && j < count && node != j;
            int64_t s = 0, d = 0;
            if (go) {
                const int ps = base + node, pd = base + j;
                const int bs = __ldg(bt + ps / a.block_size), bd = __ldg(bt + pd / a.block_size);
                if (bs < 0 || bs >= a.num_blocks || bd < 0 || bd >= a.num_blocks) {
                    if (blockIdx.y == 0) record_error(a.err, PA_DEV_BAD_BLOCK,
                                                      (long long)b * a.max_blocks +
                                                          (bs < 0 || bs >= a.num_blocks ? ps : pd) / a.block_size);
                    go = false;
                } else {
                    s = ((int64_t)bs * a.block_size + ps % a.block_size) * a.row16;
                    d = ((int64_t)bd * a.block_size + pd % a.block_size) * a.row16;
                }
            }
            const unsigned g = __ballot_sync(FULL, go);
            if (go) {
                const int at = total + __popc(g & ((1u << lane) - 1));
                src[at] = s;
                dst[at] = d;
            }
            total += __popc(g);
        }
        if (lane == 0) moves = total;
    }
    __syncthreads();
    const int nm = moves;
    if (nm == 0) return;
    const int64_t items = 2LL * a.layers * a.row16;
    for (int64_t i = (int64_t)blockIdx.y * MOVE_THREADS + threadIdx.x; i < items; i += (int64_t)gridDim.y * MOVE_THREADS) {
        const int64_t line = i / a.row16;  // layer, K or V
        const int col = (int)(i - line * a.row16);
        uint4 *c = ((line & 1) ? a.v + (line >> 1) * a.v_layer : a.k + (line >> 1) * a.k_layer) + col;
        for (int j0 = 0; j0 < nm; j0 += 8) {
            uint4 x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (j0 + e < nm) x[e] = c[src[j0 + e]];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (j0 + e < nm) c[dst[j0 + e]] = x[e];
        }
    }
}

// ---------------------------------------------------------------------------
// Verification
// ---------------------------------------------------------------------------
constexpr int V_MAX_THREADS = 512;
constexpr int V_MAX_CLUSTER = 16;
// A sequence's rows are read all at once, ahead of the walk, where a CTA's share of them
// is small (what a row costs is then latency: 32 chains of 6 nodes and 8000 logits 17.2
// us one after the other, 11.6 at once) or where they are a short drawn chain, whose
// path holds most of them, of so few sequences that each has eight CTAs at least.  Chains
// of 151936 logits, 70 % of the drafts kept, one after the other and at once: 8 x 8 32.3
// and 26.4 us, 16 x 8 32.4 and 32.6, 32 x 6 35.9 and 31.8, 64 x 6 50.5 and 49.1, 64 x 8
// 58.8 and 56.8; with four CTAs and two 128 x 6 81.7 and 85.5, 128 x 8 94.1 and 100.5,
// 256 x 8 164.8 and 185.4, as HBM then brings the rows behind a rejected draft at the cost
// of others.  All kept, 64 x 6 55.2 and 48.7, 256 x 8 187.7 and 178.5; all rejected 27.9
// and 48.7, 89.1 and 186.1.  Trees of that size have most rows off the path (64 x 8: 47.5
// us one after the other, 63.6 at once).
constexpr int64_t kAtOnceBytes = 128 << 10;
constexpr int kAtOnceChain = 8, kAtOnceCtas = 8;
constexpr float E_MIN = 1e-10f;   // the sampler's clamp of the exponential numbers

struct VerifyArgs {
    int32_t *out_tokens, *out_nodes, *out_counts;
    const void *logits;
    int64_t logits_stride;       // elements between rows
    const int32_t *tokens, *parents;
    const float *u, *noise;
    int64_t noise_stride;
    const float *temperatures;
    const float *probs;
    int64_t probs_stride;
    int32_t probs_rows;          // rows of draft_probs per sequence
    const int32_t *lens;
    int32_t batch, nodes, vocab, cluster;
    int32_t ahead;               // read the first child's row into L2 ahead of its turn
    DevError *err;
};

__device__ __forceinline__ bool better(float ka, int ia, float kb, int ib) { return ka > kb || (ka == kb && ia < ib); }

__device__ __forceinline__ uint4 ld16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Pairs of fp32.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max8(const float (&x)[8]) {
    return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), fmaxf(x[6], x[7]));
}

// A logit as it counts: NaN as -inf, +inf as the largest number.
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

template <bool FP32>
__device__ __forceinline__ float logit_at(const VerifyArgs &a, int64_t row, int i) {
    if (FP32) return tame(__ldg(static_cast<const float *>(a.logits) + row * a.logits_stride + i));
    const uint16_t h = __ldg(static_cast<const uint16_t *>(a.logits) + row * a.logits_stride + i);
    return tame(__uint_as_float((uint32_t)h << 16));
}

// Eight logits from index i on (a multiple of 8), as they stand.
template <bool FP32>
struct Raw {
    uint4 w[FP32 ? 2 : 1];
    __device__ __forceinline__ void load(const VerifyArgs &a, int64_t row, int i) {
        if (FP32) {
            const float *p = static_cast<const float *>(a.logits) + row * a.logits_stride + i;
            w[0] = ld16(p);
            w[FP32 ? 1 : 0] = ld16(p + 4);
        } else {
            w[0] = ld16(static_cast<const uint16_t *>(a.logits) + row * a.logits_stride + i);
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint4 v = w[0];
        if (FP32) {
            const uint4 t = w[FP32 ? 1 : 0];
            x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z);
            x[3] = __uint_as_float(v.w); x[4] = __uint_as_float(t.x); x[5] = __uint_as_float(t.y);
            x[6] = __uint_as_float(t.z); x[7] = __uint_as_float(t.w);
        } else {
            x[0] = bf16lo(v.x); x[1] = bf16hi(v.x); x[2] = bf16lo(v.y); x[3] = bf16hi(v.y);
            x[4] = bf16lo(v.z); x[5] = bf16hi(v.z); x[6] = bf16lo(v.w); x[7] = bf16hi(v.w);
        }
    }
};
__device__ __forceinline__ void as8(const uint4 &v, const uint4 &t, float (&x)[8]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    x[4] = __uint_as_float(t.x); x[5] = __uint_as_float(t.y); x[6] = __uint_as_float(t.z); x[7] = __uint_as_float(t.w);
}

// 2^((x - m) k) of eight logits.
__device__ __forceinline__ void powers(float (&x)[8], float m, float k) {
    const float2 nm = make_float2(-m, -m), kk = make_float2(k, k);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float2 y = mul2(add2(make_float2(x[e], x[e + 1]), nm), kk);
        x[e] = fast_exp2(y.x);
        x[e + 1] = fast_exp2(y.y);
    }
}

struct VerifyShared {
    int32_t parent[kMaxNodes], token[kMaxNodes];
    float u[kMaxNodes], x[kMaxNodes], q[kMaxNodes], p[kMaxNodes];  // of the children of the current node: logit, q, p
    float2 all[2][V_MAX_CLUSTER * V_MAX_THREADS / 32];             // the warps' values, each written into every CTA
};
// With all rows read at once: of each node maximum and sum, by warp, by CTA, and 1 / sum.
struct RowsShared {
    float2 warps[kMaxNodes][V_MAX_THREADS / 32], ctas[kMaxNodes][V_MAX_CLUSTER], rows[kMaxNodes];
};

// Reductions over the cluster.  Each warp's value goes to every CTA; two buffers in
// turn, so one barrier each: a buffer is written again only after the barrier that
// follows its last reading.  Every thread of every CTA has the same bits, as the walk
// needs (each CTA decides for itself, and they meet at the next barrier): `combine` has to
// give the same for (p, q) as for (q, p), which the two lanes of an exchange evaluate.
template <int THREADS, typename F>
__device__ __forceinline__ float2 cluster_reduce(VerifyShared &s, float2 v, int S, int rank, int &turn, float2 nothing,
                                                 F combine) {
    constexpr int W = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto warp_reduce = [&]() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            float2 t;
            t.x = __shfl_xor_sync(FULL, v.x, o);
            t.y = __shfl_xor_sync(FULL, v.y, o);
            v = combine(v, t);
        }
    };
    warp_reduce();
    float2 *mine = &s.all[turn][rank * W + warp];
    if (S == 1) {
        if (lane == 0) *mine = v;
        __syncthreads();
    } else {
        if (lane < S) {
            uint32_t dst;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_addr(mine)), "r"((uint32_t)lane));
            asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(__float_as_uint(v.x)),
                         "r"(__float_as_uint(v.y))
                         : "memory");
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    v = nothing;
    for (int i = lane; i < S * W; i += 32) v = combine(v, s.all[turn][i]);
    warp_reduce();
    turn ^= 1;
    return v;
}

// A thread's maximum and sum, of 2^((x - maximum) k).
struct Sum {
    float tm = -INFINITY, ts = 0.f;
    __device__ __forceinline__ void raise(float top, float k) {
        ts *= tm == -INFINITY ? 0.f : fast_exp2((tm - top) * k);
        tm = top;
    }
    template <bool FP32>
    __device__ __forceinline__ void add(const Raw<FP32> &w, float k) {
        float x[8];
        w.get(x);
        const float top = max8(x);  // (of the numbers among them)
        if (top > tm) raise(fminf(top, FLT_MAX), k);
        if (tm == -INFINITY) return;
        powers(x, tm, k);
        const float2 y = add2(add2(make_float2(x[0], x[1]), make_float2(x[2], x[3])),
                              add2(make_float2(x[4], x[5]), make_float2(x[6], x[7])));
        float part = y.x + y.y;
        if (!(part < INFINITY)) {  // a NaN or +inf among them
            w.get(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = tame(x[e]);
            powers(x, tm, k);
            part = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        }
        ts += part;
    }
    __device__ __forceinline__ void add(float x, float k) {
        if (x > tm) raise(x, k);
        if (tm != -INFINITY) ts += fast_exp2((x - tm) * k);
    }
};
__device__ __forceinline__ float2 join(float2 p, float2 q, float k) {
    const float mm = fmaxf(p.x, q.x), ref = mm == -INFINITY ? 0.f : mm;
    // Both products rounded: fused, p.y a + q.y b would not be what q.y b + p.y a is.
    return make_float2(mm, __fadd_rn(__fmul_rn(p.y, fast_exp2((p.x - ref) * k)), __fmul_rn(q.y, fast_exp2((q.x - ref) * k))));
}

template <bool FP32, bool PROBS, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) verify_kernel(const __grid_constant__ VerifyArgs a) {
    pdl_wait_then_release();
    __shared__ VerifyShared s;
    __shared__ RowsShared rs;
    // The cluster's CTAs have started before any of them writes into another
    // (waited for ahead of the first reduction).
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const int b = blockIdx.y, S = a.cluster, rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const bool lead = rank == 0 && tid == 0;
    const float T = __ldg(a.temperatures + b);
    int n = a.lens ? __ldg(a.lens + b) : a.nodes;
    if (tid < a.nodes) {  // (all of them: the loads need not wait for the length)
        const int64_t at = (int64_t)b * a.nodes + tid;
        const int p = a.parents ? __ldg(a.parents + at) : tid - 1, x = __ldg(a.tokens + at);
        s.u[tid] = __ldg(a.u + at);
        const bool bad_p = tid > 0 && (p < 0 || p >= tid), bad_x = tid > 0 && (x < 0 || x >= a.vocab);
        if (rank == 0 && tid < n && n <= a.nodes) {
            if (bad_p) record_error(a.err, PA_DEV_BAD_TREE, at);
            if (bad_x) record_error(a.err, PA_DEV_BAD_TOKEN, at);
        }
        s.parent[tid] = tid == 0 || tid >= n || bad_p || bad_x ? -1 : p;  // nobody's child: never kept, never subtracted
        s.token[tid] = x;
        if (rank == 0) {
            a.out_tokens[at] = -1;
            a.out_nodes[at] = -1;
        }
    }
    const bool bad_t = !(T > 1e-10f), bad_n = n < 0 || n > a.nodes;
    if (lead && bad_t && n > 0) record_error(a.err, PA_DEV_BAD_TEMPERATURE, b);  // (a padded row's may be anything)
    if (lead && bad_n) record_error(a.err, PA_DEV_BAD_CONTEXT, b);
    if (bad_n || bad_t) n = 0;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (n == 0) {  // a padded row: uniform over the cluster
        if (lead) a.out_counts[b] = 0;
        return;
    }
    const double kd = fmax(1.4426950408889634 / (double)T, 1e-37);  // log2(e) / T
    const float k = (float)kd, k_lo = (float)(kd - (double)k);
    // This CTA's chunk of a row: whole groups of 8 logits, then the ragged end.
    const int chunk = ((a.vocab + S - 1) / S + 7) & ~7;
    const int lo = min(a.vocab, rank * chunk), hi = min(a.vocab, lo + chunk);
    const int nvec = (hi - lo) / 8, tail = lo + 8 * nvec;
    const float *er = a.noise + (int64_t)b * a.noise_stride;
    int turn = 0, cur = 0, count = 1;
    float m = 0.f, inv_l = 0.f, sub = 0.f;  // of the current node: maximum, 1 / sum, S
    unsigned long long gone = 0;            // its children that were rejected (without probabilities)
    // This CTA's chunk of a row, into L2.
    auto fetch = [&](const void *p, int size) {
        const int64_t bytes = (int64_t)nvec * 8 * size;
        if (tid == 0 && bytes > 0 && bytes <= 1 << 20)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char *>(p) + (int64_t)lo * size),
                         "r"((uint32_t)bytes)
                         : "memory");
    };
    constexpr int SIZE = FP32 ? 4 : 2;
    if (a.ahead) fetch(er, 4);
    // p of a child, the exponent as a sum of two numbers.
    auto prob = [&](float x, float m, float inv_l) -> float {
        const float d = x - m, y = d * k, rest = fmaf(d, k, -y) + d * k_lo;
        const float whole = rintf(y);
        return y > -1000.f ? ldexpf(exp2f((y - whole) + rest), (int)whole) * inv_l : 0.f;
    };
    const bool chain = __syncthreads_and(tid == 0 || tid >= n || s.parent[tid] == tid - 1);
    const bool all = (int64_t)n * chunk * SIZE <= kAtOnceBytes || (PROBS && chain && n <= kAtOnceChain && S >= kAtOnceCtas);
    if (all) {
        if (tid < n && s.parent[tid] >= 0) {
            const int p = s.parent[tid], x = s.token[tid];
            s.x[tid] = logit_at<FP32>(a, (int64_t)b * a.nodes + p, x);
            s.q[tid] = PROBS ? __ldg(a.probs + ((int64_t)b * a.probs_rows + p) * a.probs_stride + x) : 1.f;
        }
        // ---- maximum and sum of every row: the warps share the rows' pieces, in order
        constexpr int W = THREADS / 32, U = FP32 ? 2 : 4, PIECE = 32 * U;  // vectors
        const int warp = tid >> 5, pieces = max(1, (nvec + PIECE - 1) / PIECE), total = n * pieces;
        for (int i = tid; i < n * W; i += THREADS) rs.warps[i / W][i % W] = make_float2(-INFINITY, 0.f);
        __syncthreads();
        const int t0 = total * warp / W, t1 = total * (warp + 1) / W;
        int node = t0 / pieces, piece = t0 - node * pieces;
        Sum sum;
        for (int t = t0; t < t1; ++t) {
            const int64_t row = (int64_t)b * a.nodes + node;
            const int v0 = piece * PIECE + lane;
            Raw<FP32> w[U];
#pragma unroll
            for (int h = 0; h < U; ++h)
                if (v0 + 32 * h < nvec) w[h].load(a, row, lo + 8 * (v0 + 32 * h));
#pragma unroll
            for (int h = 0; h < U; ++h)
                if (v0 + 32 * h < nvec) sum.add(w[h], k);
            ++piece;
            if (piece == pieces)
                for (int i = tail + lane; i < hi; i += 32) sum.add(logit_at<FP32>(a, row, i), k);
            if (piece == pieces || t + 1 == t1) {
                float2 v = make_float2(sum.tm, sum.ts);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    float2 other;
                    other.x = __shfl_xor_sync(FULL, v.x, o);
                    other.y = __shfl_xor_sync(FULL, v.y, o);
                    v = join(v, other, k);
                }
                if (lane == 0) rs.warps[node][warp] = v;
                sum = Sum();
                piece = 0;
                ++node;
            }
        }
        __syncthreads();
        if (tid < n) {
            float2 v = rs.warps[tid][0];
#pragma unroll 1
            for (int i = 1; i < W; ++i) v = join(v, rs.warps[tid][i], k);
            if (S == 1) {
                rs.ctas[tid][0] = v;
            } else {
                for (int c = 0; c < S; ++c) {
                    uint32_t dst;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst)
                                 : "r"(smem_addr(&rs.ctas[tid][rank])), "r"((uint32_t)c));
                    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(__float_as_uint(v.x)),
                                 "r"(__float_as_uint(v.y))
                                 : "memory");
                }
            }
        }
        if (S > 1) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
        if (tid < n) {
            float2 v = rs.ctas[tid][0];
            for (int c = 1; c < S; ++c) v = join(v, rs.ctas[tid][c], k);
            rs.rows[tid] = make_float2(v.x == -INFINITY ? 0.f : v.x, v.y > 0.f ? 1.f / v.y : 0.f);
        }
        __syncthreads();
        if (tid < n && s.parent[tid] >= 0) {
            const float2 r = rs.rows[s.parent[tid]];
            s.p[tid] = prob(s.x[tid], r.x, r.y);
        }
    }
    __syncthreads();
    // The sum of the probabilities of all but the rejected candidates, 16 bytes at a time.
    auto rest = [&](int64_t row) -> float {
        constexpr int N = 16 / SIZE;
        const char *r = static_cast<const char *>(a.logits) + row * a.logits_stride * SIZE;
        float acc = 0.f;
#pragma unroll 1
        for (int i = lo + N * tid; i < hi; i += N * THREADS) {
            float x[N];
            if (i + N <= hi) {
                const uint4 w = ld16(r + (int64_t)i * SIZE);
                const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < N; ++e) x[e] = tame(FP32 ? __uint_as_float(q[e % 4]) : (e & 1) ? bf16hi(q[e / 2]) : bf16lo(q[e / 2]));
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) x[e] = i + e < hi ? logit_at<FP32>(a, row, i + e) : -INFINITY;
            }
#pragma unroll 1
            for (unsigned long long g = gone; g; g &= g - 1) {
                const int at = s.token[__ffsll(g) - 1] - i;
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (at == e) x[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < N; ++e) acc += fast_exp2((x[e] - m) * k);
        }
        return cluster_reduce<THREADS>(s, make_float2(acc, 0.f), S, rank, turn, make_float2(0.f, 0.f),
                                       [](float2 p, float2 q) { return make_float2(p.x + q.x, 0.f); })
                   .x * inv_l;
    };
    while (true) {
        // ---- maximum and sum of the current node's row
        const int64_t row = (int64_t)b * a.nodes + cur;
        const float *qr = PROBS ? a.probs + ((int64_t)b * a.probs_rows + cur) * a.probs_stride : nullptr;
        const unsigned long long kids =
            (unsigned long long)__ballot_sync(FULL, lane < n && s.parent[lane] == cur) |
            (n > 32 ? (unsigned long long)__ballot_sync(FULL, lane + 32 < n && s.parent[lane + 32] == cur) << 32 : 0ull);
        if (all) {
            m = rs.rows[cur].x;
            inv_l = rs.rows[cur].y;
        } else {
            const bool kid = tid < kMaxNodes && ((kids >> tid) & 1);
            if (kid) {  // (the children's own entries, meanwhile)
                s.x[tid] = logit_at<FP32>(a, row, s.token[tid]);
                s.q[tid] = PROBS ? __ldg(qr + s.token[tid]) : 1.f;
            }
            if (a.ahead && kids)
                fetch(static_cast<const char *>(a.logits) +
                          ((int64_t)b * a.nodes + __ffsll(kids) - 1) * a.logits_stride * SIZE, SIZE);
            Sum sum;
            constexpr int U = FP32 ? 4 : 5;  // vectors under way
            for (int v0 = tid; v0 < nvec; v0 += U * THREADS) {
                Raw<FP32> w[U];
#pragma unroll
                for (int h = 0; h < U; ++h)
                    if (v0 + h * THREADS < nvec) w[h].load(a, row, lo + 8 * (v0 + h * THREADS));
#pragma unroll
                for (int h = 0; h < U; ++h) {
                    if (v0 + h * THREADS >= nvec) break;
                    sum.add(w[h], k);
                }
            }
            for (int i = tail + tid; i < hi; i += THREADS) sum.add(logit_at<FP32>(a, row, i), k);
            const float2 st = cluster_reduce<THREADS>(s, make_float2(sum.tm, sum.ts), S, rank, turn,
                                                      make_float2(-INFINITY, 0.f),
                                                      [&](float2 p, float2 q) { return join(p, q, k); });
            m = st.x == -INFINITY ? 0.f : st.x;
            inv_l = st.y > 0.f ? 1.f / st.y : 0.f;  // a row of -inf alone: every probability 0
            if (kid) s.p[tid] = prob(s.x[tid], m, inv_l);
            __syncthreads();
        }
        // ---- its children in order
        float left = 1.f, from = 1.f;  // s; what it was when it was last a sum
        sub = 0.f;
        gone = 0;
        int next = -1;
        for (unsigned long long todo = kids; todo; todo &= todo - 1) {
            const int c = __ffsll(todo) - 1;
            const float p = s.p[c], q = s.q[c];
            float w;
            if (PROBS) {
                w = fmaxf(fmaf(-sub, q, p), 0.f);
            } else {
                w = p;
                for (unsigned long long g = gone; g; g &= g - 1)
                    if (s.token[__ffsll(g) - 1] == s.token[c]) w = 0.f;  // a candidate given twice
            }
            if (s.u[c] * q * left < w) {
                next = c;
                break;
            }
            if (!PROBS) {
                left = fmaxf(left - w, 0.f);
                gone |= 1ull << c;
                // Seven bits of s lost to the difference, which is off by some 2^-23 of what it
                // was taken from: summed anew.
                if (left < from * (1.f / 128.f) && (todo & (todo - 1))) left = from = rest(row);
                continue;
            }
            sub += left;
            if (!(todo & (todo - 1))) break;  // the last child: nobody asks for s
            // s <- sum of max(p - S q, 0)
            float acc = 0.f;
            for (int v = tid; v < nvec; v += THREADS) {
                Raw<FP32> w8;
                const int i = lo + 8 * v;
                w8.load(a, row, i);
                const uint4 q0 = ld16(qr + i), q1 = ld16(qr + i + 4);
                float x[8], qq[8];
                w8.get(x);
                as8(q0, q1, qq);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = tame(x[e]);
                powers(x, m, k);
                float part = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) part += fmaxf(fmaf(-sub, qq[e], x[e] * inv_l), 0.f);
                acc += part;
            }
            for (int i = tail + tid; i < hi; i += THREADS)
                acc += fmaxf(fmaf(-sub, __ldg(qr + i), fast_exp2((logit_at<FP32>(a, row, i) - m) * k) * inv_l), 0.f);
            left = cluster_reduce<THREADS>(s, make_float2(acc, 0.f), S, rank, turn, make_float2(0.f, 0.f),
                                           [](float2 p, float2 q) { return make_float2(p.x + q.x, 0.f); })
                       .x;
        }
        if (next < 0) break;
        if (lead) {
            a.out_tokens[(int64_t)b * a.nodes + count - 1] = s.token[next];
            a.out_nodes[(int64_t)b * a.nodes + count] = next;
        }
        ++count;
        cur = next;
        if (!all) __syncthreads();  // the children's entries are written again
    }
    // ---- the last token: argmax w / E, of p / E where nothing is left of w
    const int64_t row = (int64_t)b * a.nodes + cur;
    const float *qr = PROBS && sub > 0.f ? a.probs + ((int64_t)b * a.probs_rows + cur) * a.probs_stride : nullptr;
    float key;
    int idx;
    for (int all = 0;; ++all) {
        if (all) {
            sub = 0.f;
            qr = nullptr;
            gone = 0;
        }
        key = 0.f;
        idx = 0x7fffffff;
        auto offer = [&](float r, int i) {  // i ascends: the first of equals stays
            if (!(r > key)) return;
            if (!PROBS)
                for (unsigned long long g = gone; g; g &= g - 1)
                    if (s.token[__ffsll(g) - 1] == i) return;
            key = r;
            idx = i;
        };
        constexpr int U = FP32 || PROBS ? 1 : 2;
        for (int v0 = tid; v0 < nvec; v0 += U * THREADS) {
            Raw<FP32> w[U];
            uint4 e0[U], e1[U], q0[U], q1[U];
#pragma unroll
            for (int h = 0; h < U; ++h) {
                const int i = lo + 8 * (v0 + h * THREADS);
                if (v0 + h * THREADS >= nvec) break;
                w[h].load(a, row, i);
                e0[h] = ld16(er + i);
                e1[h] = ld16(er + i + 4);
                if (PROBS && qr) {
                    q0[h] = ld16(qr + i);
                    q1[h] = ld16(qr + i + 4);
                }
            }
#pragma unroll
            for (int h = 0; h < U; ++h) {
                if (v0 + h * THREADS >= nvec) break;
                float x[8], ee[8], qq[8];
                w[h].get(x);
                as8(e0[h], e1[h], ee);
                powers(x, m, k);
                // NaN (of a NaN logit, or +inf less the largest number): out of the question
                // but for the latter, which counts as the maximum.
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!(x[e] < INFINITY)) {
                        float y[8];
                        w[h].get(y);
                        x[e] = fast_exp2((tame(y[e]) - m) * k);
                    }
                if (PROBS && qr) {
                    as8(q0[h], q1[h], qq);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = fmaf(-sub, qq[e], x[e] * inv_l);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __fdividef(x[e], fmaxf(ee[e], E_MIN));
                if (max8(x) > key)
#pragma unroll
                    for (int e = 0; e < 8; ++e) offer(x[e], lo + 8 * (v0 + h * THREADS) + e);
            }
        }
        for (int i = tail + tid; i < hi; i += THREADS) {
            float w = fast_exp2((logit_at<FP32>(a, row, i) - m) * k);
            if (PROBS && qr) w = fmaf(-sub, __ldg(qr + i), w * inv_l);
            offer(__fdividef(w, fmaxf(__ldg(er + i), E_MIN)), i);
        }
        const float2 r = cluster_reduce<THREADS>(s, make_float2(key, __int_as_float(idx)), S, rank, turn,
                                                 make_float2(0.f, __int_as_float(0x7fffffff)), [](float2 p, float2 q) {
                                                     return better(q.x, __float_as_int(q.y), p.x, __float_as_int(p.y)) ? q : p;
                                                 });
        key = r.x;
        idx = __float_as_int(r.y);
        if (key > 0.f || all || (sub == 0.f && gone == 0)) break;  // uniform over the cluster
    }
    if (lead) {
        a.out_tokens[(int64_t)b * a.nodes + count - 1] = idx == 0x7fffffff ? 0 : idx;
        a.out_nodes[(int64_t)b * a.nodes] = 0;
        a.out_counts[b] = count;
    }
}

// CTAs per sequence: as many as leave all sequences room to run at once (1024
// threads per SM, with a tenth to spare for clusters that do not fit), at most 8 and
// 2048 logits a CTA at least; 16 (no portable size) for up to four sequences, where one
// SM's loads and exponentials are what a row waits for (1 x 6 x 151936: 17.4 us with
// 8, 14.9 with 16; 4 x 32: 20.1 and 16.5; but 8 x 32: 26.0 and 27.7).
int ctas_per_seq(int batch, int vocab, int sms) {
    int S = 1;
    if (32LL * batch <= sms && vocab / 16 >= 2048) return V_MAX_CLUSTER;
    while (S < 8 && 20LL * batch * S <= 36LL * sms && vocab / (2 * S) >= 2048) S *= 2;
    return S;
}

template <bool FP32, bool PROBS, int THREADS>
pa_status launch_verify(VerifyArgs &a, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.cluster, (unsigned)a.batch);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (a.cluster > 8) {
        // Allowed once per (device, variant), which takes 3 us, and the device asked whether
        // it can run such a cluster: where its SMs lie in smaller groups (a partitioned
        // device) the portable size serves.
        static std::atomic<int> known[64];  // 0: not asked, 1: it can, 2: it cannot
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
        if (dev < 0 || dev >= 64) return fail(PA_ERR_UNSUPPORTED, "device %d", dev);
        int can = known[dev].load(std::memory_order_acquire);
        if (can == 0) {
            int clusters = 0;
            cfg.numAttrs = 1;
            e = cudaFuncSetAttribute(verify_kernel<FP32, PROBS, THREADS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, verify_kernel<FP32, PROBS, THREADS>, &cfg);
            cfg.numAttrs = 2;
            if (e != cudaSuccess) (void)cudaGetLastError();
            can = e == cudaSuccess && clusters > 0 ? 1 : 2;
            known[dev].store(can, std::memory_order_release);
        }
        if (can == 2) {
            a.cluster = 8;
            cfg.gridDim.x = attr[0].val.clusterDim.x = 8;
        }
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<FP32, PROBS, THREADS>, a);
    if (e != cudaSuccess) return cuda_fail(e, "verify_kernel");
    return check_launch("verify_kernel");
}

template <bool FP32, bool PROBS>
pa_status launch_verify(VerifyArgs &a, cudaStream_t stream) {
    const int sms = sm_count();
    a.cluster = ctas_per_seq(a.batch, a.vocab, sms);
    // A row read ahead in vain costs more than the wait it saves once the sequences fill
    // the GPU (64 sequences 52 us without, 56 with; 32 trees of 12 nodes 39.5 and 38.3; 16
    // sequences 28.8 and 27.3).
    a.ahead = 8LL * a.batch <= 2LL * sms;
    // Few CTAs: twice the threads.
    const bool few = (int64_t)a.batch * a.cluster <= 2LL * sms;
    return few ? launch_verify<FP32, PROBS, 512>(a, stream) : launch_verify<FP32, PROBS, 256>(a, stream);
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_tree_metadata(int64_t *tree_mask, int32_t *positions, int32_t *slot_mapping, const int32_t *parents,
                           const int32_t *context_lens, const int32_t *draft_lens, const int32_t *block_tables,
                           int32_t max_blocks_per_seq, int32_t batch, int32_t num_drafts, int32_t block_size,
                           pa_stream_t stream) {
    using namespace pa;
    if (batch < 0) return fail(PA_ERR_INVALID_ARG, "batch < 0");
    if (num_drafts <= 0) return fail(PA_ERR_INVALID_ARG, "num_drafts must be positive");
    if (num_drafts > kMaxNodes) return fail(PA_ERR_UNSUPPORTED, "%d drafts (at most %d)", num_drafts, kMaxNodes);
    if (batch == 0) return PA_OK;
    if (!tree_mask || !positions || !slot_mapping || !context_lens || !block_tables)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (block_size <= 0 || max_blocks_per_seq <= 0)
        return fail(PA_ERR_INVALID_ARG, "block_size and max_blocks_per_seq must be positive");
    if (reinterpret_cast<uintptr_t>(tree_mask) & 7u) return fail(PA_ERR_INVALID_ARG, "tree_mask must be 8-byte aligned");
    MetaArgs a = {reinterpret_cast<unsigned long long *>(tree_mask), positions, slot_mapping, parents, context_lens,
                  draft_lens, block_tables, max_blocks_per_seq, batch, num_drafts, block_size, device_error_ptr()};
    const int64_t grid = ((int64_t)batch * num_drafts + 127) / 128;
    return launch_pdl(tree_metadata_kernel, dim3((unsigned)grid), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream),
                      "tree_metadata_kernel", a);
}

pa_status pa_verify_drafts(int32_t *out_tokens, int32_t *out_nodes, int32_t *out_counts, const void *logits,
                           int64_t logits_row_stride, int32_t logits_is_fp32, const int32_t *tokens,
                           const int32_t *parents, const float *uniforms, const float *exp_noise,
                           int64_t noise_row_stride, const float *temperatures, const float *draft_probs,
                           int64_t probs_row_stride, int32_t probs_rows, const int32_t *draft_lens, int32_t batch,
                           int32_t num_nodes, int32_t vocab, pa_stream_t stream) {
    using namespace pa;
    if (batch < 0 || vocab < 0) return fail(PA_ERR_INVALID_ARG, "negative size");
    if (num_nodes <= 0) return fail(PA_ERR_INVALID_ARG, "num_nodes must be positive");
    if (num_nodes > kMaxNodes) return fail(PA_ERR_UNSUPPORTED, "%d nodes (at most %d)", num_nodes, kMaxNodes);
    if (batch == 0) return PA_OK;
    if (vocab == 0) return fail(PA_ERR_INVALID_ARG, "vocab must be positive");
    if (vocab > (1 << 30)) return fail(PA_ERR_UNSUPPORTED, "vocab %d (at most 2^30)", vocab);
    if (batch > 65535) return fail(PA_ERR_UNSUPPORTED, "batch %d (at most 65535 sequences per call)", batch);
    if (!out_tokens || !out_nodes || !out_counts || !logits || !tokens || !uniforms || !exp_noise || !temperatures)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (logits_is_fp32 != 0 && logits_is_fp32 != 1) return fail(PA_ERR_INVALID_ARG, "logits_is_fp32 must be 0 or 1");
    const int align = logits_is_fp32 ? 4 : 8;
    if (logits_row_stride < vocab || logits_row_stride % align)
        return fail(PA_ERR_INVALID_ARG, "logits_row_stride must be >= vocab and a multiple of %d", align);
    if (noise_row_stride < vocab || noise_row_stride % 4)
        return fail(PA_ERR_INVALID_ARG, "noise_row_stride must be >= vocab and a multiple of 4");
    if (draft_probs) {
        if (probs_row_stride < vocab || probs_row_stride % 4)
            return fail(PA_ERR_INVALID_ARG, "probs_row_stride must be >= vocab and a multiple of 4");
        if (probs_rows < num_nodes - 1)
            return fail(PA_ERR_INVALID_ARG, "draft_probs has %d rows a sequence, at least num_nodes - 1 are needed", probs_rows);
    }
    if (!aligned16(logits) || !aligned16(exp_noise) || !aligned16(draft_probs))
        return fail(PA_ERR_INVALID_ARG, "logits, exp_noise and draft_probs must be 16-byte aligned");
    if (sm_count() <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    VerifyArgs a = {out_tokens, out_nodes, out_counts, logits, logits_row_stride, tokens, parents, uniforms, exp_noise,
                    noise_row_stride, temperatures, draft_probs, probs_row_stride, probs_rows, draft_lens, batch,
                    num_nodes, vocab, 1, 0, device_error_ptr()};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (logits_is_fp32) return draft_probs ? launch_verify<true, true>(a, s) : launch_verify<true, false>(a, s);
    return draft_probs ? launch_verify<false, true>(a, s) : launch_verify<false, false>(a, s);
}

pa_status pa_compact_kvcache(void *k_cache, int64_t k_layer_stride, void *v_cache, int64_t v_layer_stride,
                             const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *context_lens,
                             const int32_t *draft_lens, const int32_t *nodes, const int32_t *counts, int32_t batch,
                             int32_t num_nodes, int32_t num_layers, int32_t num_kv_heads, int32_t head_dim,
                             int32_t block_size, int32_t num_blocks, pa_stream_t stream) {
    using namespace pa;
    if (batch < 0 || num_layers < 0) return fail(PA_ERR_INVALID_ARG, "negative size");
    if (num_nodes <= 0) return fail(PA_ERR_INVALID_ARG, "num_nodes must be positive");
    if (num_nodes > kMaxNodes) return fail(PA_ERR_UNSUPPORTED, "%d nodes (at most %d)", num_nodes, kMaxNodes);
    if (batch == 0 || num_layers == 0) return PA_OK;
    if (!k_cache || !v_cache || !block_tables || !context_lens || !nodes || !counts)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (num_kv_heads <= 0 || head_dim <= 0) return fail(PA_ERR_INVALID_ARG, "bad head shape");
    if (head_dim != 128) return fail(PA_ERR_UNSUPPORTED, "head_dim %d (only 128)", head_dim);
    if (num_kv_heads > (1 << 20)) return fail(PA_ERR_UNSUPPORTED, "too many heads");
    if (block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "block_size, max_blocks_per_seq and num_blocks must be positive");
    if (num_layers > 1 && (k_layer_stride % 8 || v_layer_stride % 8 || k_layer_stride <= 0 || v_layer_stride <= 0))
        return fail(PA_ERR_INVALID_ARG, "layer strides must be positive multiples of 8 elements");
    if (!aligned16(k_cache) || !aligned16(v_cache)) return fail(PA_ERR_INVALID_ARG, "caches must be 16-byte aligned");
    const int sms = sm_count();
    if (sms <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    MoveArgs a = {static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), k_layer_stride / 8, v_layer_stride / 8,
                  block_tables, context_lens, draft_lens, nodes, counts, max_blocks_per_seq, batch, num_nodes, num_layers,
                  num_kv_heads * 16, block_size, num_blocks, device_error_ptr()};
    // One item a thread while the CTAs fit the GPU together (eight per SM), more after that.
    const int64_t items = 2LL * num_layers * a.row16;
    const int64_t y = std::max<int64_t>(1, std::min<int64_t>((items + MOVE_THREADS - 1) / MOVE_THREADS,
                                                             std::min<int64_t>(65535, 8LL * sms / batch)));
    return launch_pdl(compact_kernel, dim3((unsigned)batch, (unsigned)y), dim3(MOVE_THREADS), 0,
                      reinterpret_cast<cudaStream_t>(stream), "compact_kernel", a);
}

}  // extern "C"
