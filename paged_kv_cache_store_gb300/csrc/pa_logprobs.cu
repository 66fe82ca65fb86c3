// pa_logprobs.cu -- log probabilities of given tokens, entropy, top alternatives.
//
// What it computes, per row of logits x with temperature T (z = x / T):
//   lse = ln sum_i e^{z_i},  logprob(i) = z_i - lse,
//   entropy = lse - sum_i p_i z_i  (p = softmax z),
//   the k largest logits in order, the lower index first among equals.
//
// How (GB300 design): a row is split over the CTAs of a thread-block cluster
// (one CTA when there are many rows) and read from HBM once.
//  * Sums: each thread keeps a reference m and S = sum 2^y, E = sum 2^y y with
//    y = (x - m) * log2(e) / T, in fp32 pairs (packed add, mul and fma), one
//    ex2 per element.  m is in logit units and y a product of a difference, so
//    rows of the type's lowest value or of very large logits do not overflow.
//    m only moves when a logit exceeds it by 32 in base 2.  Threads, warps
//    and CTAs combine as (m, S, E) triples.
//  * Top k: a thread also keeps the largest logit it has seen, the vector (8
//    logits) that first held it, and the largest of each eighth of its
//    vectors.  The threads form 64 groups, by lane and the warp's parity; the
//    k-th largest of the groups' maxima, with its vector as the tie-break, is
//    a threshold that at least k entries of the CTA's chunk reach.  The
//    eighths whose maximum reaches it are listed and re-read by all threads,
//    which collect the entries that do: for logits in random order 5 of them
//    at k = 5, 24 at 20 and 44 at 32.  (Re-reading a thread's whole share cost
//    42 % more DRAM traffic: a row has left L2 by then.  Re-reading by the
//    owners alone cost 13 us a row: a warp's lanes had different eighths to
//    wait for.)  The collected keys (logit, then index) are ranked by
//    counting.  A chunk with more than CAP such entries, or with NaNs that hid
//    some, is selected by k passes of a plain maximum instead.
//    The CTAs' lists meet in the cluster's first CTA, where an entry's rank is
//    its place in its own list plus the entries above it in the others'.
#include <math.h>

#include <algorithm>

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int LP_MAX_CLUSTER = 8;
constexpr int LP_MAX_TOP = 32;
constexpr int LP_SEGS = 8;        // parts of a thread's vectors with a maximum of their own
constexpr float LP_LAZY = 32.f;   // log2 headroom before the reference moves
constexpr float LP_FLOOR = -200.f;  // 2^-200 is 0: keeps 0 * y finite for y = -inf
constexpr unsigned FULL = 0xffffffffu;
typedef unsigned long long u64;

struct LpArgs {
    float *logprobs, *entropy;
    int32_t *top_ids;
    float *top_logprobs;
    const void *logits;
    int64_t stride;
    const float *temperatures;  // null: 1
    const int32_t *tokens;
    int32_t vocab, top, cluster;
    DevError *err;
};

// (m, S, E) of a set of logits; m = -inf when it holds nothing finite.
struct Stat {
    float m, s, e;
};

// A float as an unsigned integer in the same order (-0 as +0); NaN lowest.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return x != x ? 0u : (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
    return o == 0 ? NAN : __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o);
}
// Larger logits first, then lower indices (or vectors).  0: nothing.
__device__ __forceinline__ u64 key_of(float x, uint32_t i) { return ((u64)ordered(x) << 32) | (uint32_t)~i; }

__device__ __forceinline__ uint4 ld16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Packed pairs of fp32.
__device__ __forceinline__ u64 pack2(float a, float b) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(u64 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // keeps a NaN
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {  // drops a NaN
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight consecutive logits.
template <bool FP32>
struct Vec {
    uint4 a, b;  // b: fp32 only
    __device__ __forceinline__ void load(const void *row, int i) {
        const char *p = static_cast<const char *>(row) + (int64_t)i * (FP32 ? 4 : 2);
        a = ld16(p);
        if (FP32) b = ld16(p + 16);
    }
    // The pair of logits 2j, 2j+1.
    __device__ __forceinline__ void pair(int j, float &x, float &y) const {
        if (FP32) {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            x = __uint_as_float(w[2 * j]);
            y = __uint_as_float(w[2 * j + 1]);
        } else {
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
            x = bf16lo(w[j]);
            y = bf16hi(w[j]);
        }
    }
    __device__ __forceinline__ float top() const {  // the largest, NaNs dropped
        if (FP32) {
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x, y;
                pair(j, x, y);
                m = fmaxf(m, fmaxf(x, y));
            }
            return m;
        }
        const uint32_t w = max_bf16x2(max_bf16x2(a.x, a.y), max_bf16x2(a.z, a.w));
        return fmaxf(bf16lo(w), bf16hi(w));
    }
};

template <bool FP32>
__device__ __forceinline__ float logit(const void *row, int i) {
    if (FP32) return __ldg(static_cast<const float *>(row) + i);
    return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t *>(row) + i) << 16);
}

// A thread's running state over its vectors.
struct Run {
    float m, limit;   // reference, and the logit above which it moves
    u64 s, e;         // packed pairs
    float top;        // largest logit so far and the vector that first held it
    uint32_t top_vec; // 0xffffffff: none
};

__device__ __forceinline__ void move_reference(Run &r, float to, float kk) {
    if (r.m != -INFINITY) {
        float s0, s1, e0, e1;
        unpack2(r.s, s0, s1);
        unpack2(r.e, e0, e1);
        const float d = fmaxf((r.m - to) * kk, LP_FLOOR), f = fast_exp2(d);
        r.s = pack2(s0 * f, s1 * f);
        r.e = pack2((e0 + s0 * d) * f, (e1 + s1 * d) * f);
    }
    r.m = to;
    r.limit = to + LP_LAZY / kk;
}

// Adds a pair's weights to s and weighted exponents to e (a lone logit: its
// partner is -inf).  The floor keeps 0 * y finite for y = -inf.
__device__ __forceinline__ void add_pair(u64 &s, u64 &e, float x, float y, u64 negm, u64 kk2) {
    float a, b;
    unpack2(mul2(add2(pack2(x, y), negm), kk2), a, b);
    a = max_nan(a, LP_FLOOR);
    b = max_nan(b, LP_FLOOR);
    const u64 ex = pack2(fast_exp2(a), fast_exp2(b));
    s = add2(s, ex);
    e = fma2(ex, pack2(a, b), e);
}

// The reference, negated, as a pair; moved first if t exceeds its limit.
__device__ __forceinline__ u64 reference(Run &r, float t, float kk) {
    if (t > r.limit) move_reference(r, t, kk);
    const float nm = r.m == -INFINITY ? 0.f : -r.m;
    return pack2(nm, nm);
}

// A batch of vectors (the first n of them) into the sums; returns the largest
// logit.  The batch has sums of its own, so that the running ones take one
// rounding a batch.
template <int THREADS, bool FP32, int N>
__device__ __forceinline__ float take(Run &r, const Vec<FP32> (&v)[N], int n, int vec0, float kk, u64 kk2) {
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < N; ++u)
        if (u < n) {
            const float t = v[u].top();
            if (t > r.top) {
                r.top = t;
                r.top_vec = (uint32_t)(vec0 + u * THREADS);
            }
            top = fmaxf(top, t);
        }
    const u64 negm = reference(r, top, kk);
    u64 s = pack2(0.f, 0.f), e = s;
#pragma unroll
    for (int u = 0; u < N; ++u)
        if (u < n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float p, q;
                v[u].pair(j, p, q);
                add_pair(s, e, p, q, negm, kk2);
            }
        }
    r.s = add2(r.s, s);
    r.e = add2(r.e, e);
    return top;
}

// The largest 64-bit key of a warp, word by word.
__device__ __forceinline__ u64 warp_max(u64 k) {
    const uint32_t hi = (uint32_t)(k >> 32), m = __reduce_max_sync(FULL, hi);
    return ((u64)m << 32) | __reduce_max_sync(FULL, hi == m ? (uint32_t)k : 0u);
}

// Joins the lanes' statistics; every lane holds the same bits afterwards.
__device__ __forceinline__ Stat warp_join(Stat a, float kk) {
    const float m = from_ordered(__reduce_max_sync(FULL, ordered(a.m)));
    if (a.m != m && a.s != 0.f) {
        const float d = fmaxf((a.m - m) * kk, LP_FLOOR), f = fast_exp2(d);
        a.e = (a.e + a.s * d) * f;
        a.s *= f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(FULL, a.s, o);
        a.e += __shfl_xor_sync(FULL, a.e, o);
    }
    return Stat{m, a.s, a.e};
}

template <bool FP32, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprobs_kernel(const LpArgs a) {
    constexpr int WARPS = THREADS / 32;
    constexpr int CAP = 4 * THREADS;  // collected entries of a chunk
    pdl_wait_then_release();
    // Distributed shared memory is written only once every CTA of the cluster runs.
    if (a.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    __shared__ u64 buf[CAP];
    __shared__ float seg_top[LP_SEGS][THREADS];
    __shared__ u64 group[WARPS][32];
    __shared__ Stat stats[WARPS];
    __shared__ uint16_t items[LP_SEGS * THREADS];  // segment, thread
    __shared__ int count, nitems;
    __shared__ u64 threshold;
    __shared__ u64 lists[LP_MAX_CLUSTER][LP_MAX_TOP];  // in the cluster's first CTA
    __shared__ Stat cstats[LP_MAX_CLUSTER];            // likewise
    __shared__ u64 mine[LP_MAX_TOP];
    constexpr int UNROLL = FP32 ? 2 : 4;  // vectors of a thread in flight (64 bytes)
    constexpr int BATCH = UNROLL * THREADS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = a.cluster;
    const int64_t row = blockIdx.x / (unsigned)S;
    const int rank = (int)(blockIdx.x % (unsigned)S);
    const float T = a.temperatures ? __ldg(a.temperatures + row) : 1.f;
    const bool bad_t = !(T > 1e-10f);
    // (At least the smallest fp32 number: under T = inf, -inf stays -inf and every
    // finite difference has weight 1.)
    const float kk = bad_t ? 1.f : fmaxf(1.4426950408889634f / T, 0x1p-149f);
    const char *x = static_cast<const char *>(a.logits) + row * a.stride * (FP32 ? 4 : 2);
    // This CTA's chunk of the row, a multiple of 8 logits except at the end.
    const int chunk = (int)((((int64_t)a.vocab + S - 1) / S + 7) & ~7ll);
    const int lo = (int)min((int64_t)a.vocab, (int64_t)rank * chunk), hi = (int)min((int64_t)a.vocab, (int64_t)lo + chunk);
    const int nvec = (hi - lo) / 8;
    if (tid < LP_MAX_TOP) mine[tid] = 0;
    if (tid == 0) {
        count = nitems = 0;
        threshold = 0;
    }
    // The given token's logit, ahead of its use.
    const bool answers = rank == 0 && tid == THREADS - 1;
    const int32_t tok = answers ? __ldg(a.tokens + row) : -1;
    const float tok_logit = tok >= 0 && tok < a.vocab ? logit<FP32>(x, tok) : 0.f;

    // ---- one pass: sums, and the largest logits
    Run r;
    r.m = r.limit = r.top = -INFINITY;
    r.s = r.e = pack2(0.f, 0.f);
    // A thread's first vector stands for -inf until it sees more than that.
    r.top_vec = tid < nvec ? (uint32_t)tid : 0xffffffffu;
    const u64 kk2 = pack2(kk, kk);
    auto fetch = [&](Vec<FP32>(&v)[UNROLL], int i) {  // batch i; a repeat past the end is ignored later
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) v[u].load(x, lo + 8 * min(i * BATCH + tid + u * THREADS, nvec - 1));
    };
    // Batches of a segment; segment s holds batches [s * per, (s + 1) * per).
    const int batches = (nvec + BATCH - 1) / BATCH, per = (batches + LP_SEGS - 1) / LP_SEGS;
    {
        Vec<FP32> v[UNROLL];
        if (batches > 0) fetch(v, 0);
        float top = -INFINITY;
        int left = per, seg = 0;
        for (int i = 0; i < batches; ++i) {
            const int v0 = i * BATCH + tid;
            Vec<FP32> next[UNROLL];
            if (i + 1 < batches) fetch(next, i + 1);
            if ((i + 1) * BATCH <= nvec) {  // (without a test per vector: 204 us instead of 216 for 4096 rows)
                top = fmaxf(top, take<THREADS, FP32>(r, v, UNROLL, v0, kk, kk2));
            } else if (v0 < nvec) {
                top = fmaxf(top, take<THREADS, FP32>(r, v, (nvec - v0 + THREADS - 1) / THREADS, v0, kk, kk2));
            }
            if (--left == 0 || i + 1 == batches) {
                if (a.top > 0) seg_top[seg][tid] = top;
                top = -INFINITY;
                left = per;
                ++seg;
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) v[u] = next[u];
        }
    }
    // The ragged end of the row: one logit per thread, each a vector of its own
    // number (after the others, in order), so that equal ones have distinct keys.
    const int tail = lo + 8 * nvec + tid;
    float tail_logit = 0.f;
    if (tail < hi) {
        tail_logit = logit<FP32>(x, tail);
        if (tail_logit > r.top || r.top_vec == 0xffffffffu) {
            r.top = tail_logit != tail_logit ? -INFINITY : tail_logit;
            r.top_vec = (uint32_t)(nvec + tid);
        }
        add_pair(r.s, r.e, tail_logit, -INFINITY, reference(r, tail_logit, kk), kk2);
    }
    // References become the largest logits themselves: ln of the final sum is
    // then small where one entry holds the row, and exact to fp32.
    if (r.top > r.m) move_reference(r, r.top, kk);
    {
        float s0, s1, e0, e1;
        unpack2(r.s, s0, s1);
        unpack2(r.e, e0, e1);
        const Stat st = warp_join(Stat{r.m, s0 + s1, e0 + e1}, kk);
        if (lane == 0) stats[warp] = st;
    }

    // ---- the chunk's k largest, in order, in mine[]
    if (a.top > 0) {
        const int want = min(a.top, hi - lo);
        const u64 own = r.top_vec == 0xffffffffu ? 0ull : key_of(r.top, r.top_vec);
        group[warp][lane] = own;
        __syncthreads();
        u64 g0 = group[0][lane], g1 = group[1][lane];  // even and odd warps' lanes
#pragma unroll
        for (int w = 2; w < WARPS; w += 2) {
            g0 = max(g0, group[w][lane]);
            g1 = max(g1, group[w + 1][lane]);
        }
        // Each warp ranks its share of the 64 groups; keys are distinct but for 0 (an
        // empty group), which the threshold is if fewer than k groups hold any.
        constexpr int SHARE = 32 / WARPS;
#pragma unroll 8
        for (int j = 0; j < 2 * SHARE; ++j) {
            const u64 k = __shfl_sync(FULL, j < SHARE ? g0 : g1, warp * SHARE + j % SHARE);
            const int above = __popc(__ballot_sync(FULL, g0 > k)) + __popc(__ballot_sync(FULL, g1 > k));
            if (above == a.top - 1 && lane == 0) threshold = k;
        }
        __syncthreads();
        const u64 thr = threshold;
        auto collect = [&](float t, uint32_t vec, int i) {
            if (key_of(t, vec) >= thr) {
                const int at = atomicAdd(&count, 1);
                if (at < CAP) buf[at] = key_of(t, (uint32_t)i);
            }
        };
        if (own != 0 && own >= thr) {
            const float thr_top = thr >> 32 ? from_ordered((uint32_t)(thr >> 32)) : -INFINITY;
            for (int seg = 0; seg * per < batches; ++seg)
                if (seg_top[seg][tid] >= thr_top) items[atomicAdd(&nitems, 1)] = (uint16_t)(seg * THREADS + tid);
            if (tail < hi) collect(tail_logit, (uint32_t)(nvec + tid), tail);
        }
        __syncthreads();
        // An item's vectors: segment's batches, UNROLL of the thread's in each.
        const int vecs = per * UNROLL, work = nitems * vecs;
        for (int w0 = tid; w0 < work; w0 += 2 * THREADS) {
            Vec<FP32> v[2];
            int at[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int w = w0 + u * THREADS;
                at[u] = nvec;
                if (w < work) {
                    const int item = w / vecs, j = w - item * vecs;
                    at[u] = (items[item] / THREADS * per + j / UNROLL) * BATCH + j % UNROLL * THREADS +
                            items[item] % THREADS;
                }
                if (at[u] < nvec) v[u].load(x, lo + 8 * at[u]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (at[u] >= nvec || key_of(v[u].top(), (uint32_t)at[u]) < thr) continue;
                float t[8];
                unsigned hit = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[u].pair(j, t[2 * j], t[2 * j + 1]);
#pragma unroll
                for (int j = 0; j < 8; ++j) hit |= (key_of(t[j], (uint32_t)at[u]) >= thr ? 1u : 0u) << j;
                int to = atomicAdd(&count, __popc(hit));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (hit >> j & 1) {
                        if (to < CAP) buf[to] = key_of(t[j], (uint32_t)(lo + 8 * at[u] + j));
                        ++to;
                    }
            }
        }
        __syncthreads();
        const int n = count;
        if (n >= want && n <= CAP) {
            for (int i = tid; i < n; i += THREADS) {
                const u64 k = buf[i];
                int above = 0;
                int j = 0;
                for (; j + 8 <= n; j += 8)
#pragma unroll
                    for (int u = 0; u < 8; ++u) above += buf[j + u] > k;
                for (; j < n; ++j) above += buf[j] > k;
                if (above < want) mine[above] = k;
            }
        } else {  // k passes: the largest key below the last one
            u64 last = ~0ull;
            for (int i = 0; i < want; ++i) {
                u64 best = 0;
                for (int e = lo + tid; e < hi; e += THREADS) {
                    const u64 k = key_of(logit<FP32>(x, e), (uint32_t)e);
                    if (k < last && k > best) best = k;
                }
                best = warp_max(best);
                __syncthreads();
                if (lane == 0) group[0][warp] = best;
                __syncthreads();
                best = group[0][0];
#pragma unroll
                for (int w = 1; w < WARPS; ++w) best = max(best, group[0][w]);
                if (tid == 0) mine[i] = best;
                last = best;
            }
        }
    }
    __syncthreads();
    // ---- the CTA's statistics (each warp joins them), to the cluster's first CTA
    Stat all = warp_join(lane < WARPS ? stats[lane] : Stat{-INFINITY, 0.f, 0.f}, kk);
    if (S > 1) {
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (tid < a.top) {
            uint32_t dst;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_addr(&lists[rank][tid])), "r"(0u));
            asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(dst), "l"(mine[tid]) : "memory");
        }
        if (tid >= 32 && tid < 35) {
            const int f = tid - 32;
            uint32_t dst;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(smem_addr(&cstats[rank])), "r"(0u));
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(dst + 4 * f),
                         "r"(__float_as_uint(f == 0 ? all.m : f == 1 ? all.s : all.e))
                         : "memory");
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank != 0) return;
        all = warp_join(lane < S ? cstats[lane] : Stat{-INFINITY, 0.f, 0.f}, kk);
    }
    // ---- the row's answers
    const float lsum = logf(all.s);
    auto logprob = [&](float t) -> float {
        // A row without a finite logit; a logit of probability 0 (also where T is inf).
        if (all.s == 0.f || (t == -INFINITY && all.s == all.s)) return -INFINITY;
        return (t - all.m) / T - lsum;
    };
    if (answers) {
        float lp = -INFINITY;
        if (bad_t) {
            record_error(a.err, PA_DEV_BAD_TEMPERATURE, row);
            lp = NAN;
        } else if (tok >= a.vocab) {
            record_error(a.err, PA_DEV_BAD_TOKEN, row);
        } else if (tok >= 0) {
            lp = logprob(tok_logit);
        }
        a.logprobs[row] = lp;
        a.entropy[row] = bad_t ? NAN : all.s == 0.f ? 0.f : lsum - 0.6931471805599453f * (all.e / all.s);
    }
    for (int i = tid; i < S * a.top; i += THREADS) {
        const int c = i / a.top, at = i - c * a.top;
        const u64 k = S > 1 ? lists[c][at] : mine[at];
        if (k == 0) continue;
        int place = at;
        if (S > 1) {  // the entries above k in the other lists, searched side by side
            int pos[LP_MAX_CLUSTER];
#pragma unroll
            for (int o = 0; o < LP_MAX_CLUSTER; ++o) pos[o] = 0;
            for (int step = 1 << (31 - __clz(a.top)); step > 0; step >>= 1)
#pragma unroll
                for (int o = 0; o < LP_MAX_CLUSTER; ++o)
                    if (o < S && pos[o] + step <= a.top && lists[o][pos[o] + step - 1] > k) pos[o] += step;
            place = 0;  // (its own list counts the entries before it)
#pragma unroll
            for (int o = 0; o < LP_MAX_CLUSTER; ++o) place += pos[o];
        }
        if (place < a.top) {
            a.top_ids[row * a.top + place] = bad_t ? -1 : (int32_t)~(uint32_t)k;
            a.top_logprobs[row * a.top + place] = bad_t ? NAN : logprob(from_ordered((uint32_t)(k >> 32)));
        }
    }
}

// CTAs per row: the largest power of two with which the rows' CTAs run at once
// (four of 256 threads per SM), at most 8 (a portable cluster) and at least 2048
// logits per CTA.  One step more costs a second wave and a cluster's barriers:
// 256 rows of 151936 28 us with four CTAs a row, 22.5 with two; 512 rows of 8000
// 13.7 with two, 7.7 with one.
int lp_ctas_per_row(int rows, int vocab, int sms) {
    int S = 1;
    while (S < LP_MAX_CLUSTER && (int64_t)rows * 2 * S <= 4LL * sms && vocab / (2 * S) >= 2048) S *= 2;
    return S;
}

// Threads per CTA.  A CTA streams its chunk, then goes through the selection's
// phases, some 5 us whatever the chunk; with CTAs of 128 threads twice as many
// rows are on their way.  That pays where rows wait for a CTA (4096 rows of 500
// logits 22.6 us instead of 35.3, of 32000 60.6 instead of 68.8; of 50257 no
// difference; of 151936 205 instead of 204, with 32 alternatives 257 instead of
// 228) and for short chunks that fill the GPU once (512 rows of 8000 7.1 instead
// of 7.7, of 32000 20.0 instead of 17.2 in fp32), not for few rows (40 of 4000
// 5.2 instead of 5.0).  With 64 threads nothing was faster than with 128.
int lp_threads(int64_t ctas, int chunk, int sms) {
    const int most = ctas > 4LL * sms ? 40960 : ctas > 2LL * sms ? 8192 : 0;
    return chunk <= most ? 128 : 256;
}

template <bool FP32, int THREADS>
pa_status launch_logprobs(const LpArgs &a, int32_t rows, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.cluster * (unsigned)rows);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, logprobs_kernel<FP32, THREADS>, a);
    if (e != cudaSuccess) return cuda_fail(e, "logprobs_kernel");
    return check_launch("logprobs_kernel");
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_logprobs(float *logprobs, float *entropy, int32_t *top_ids, float *top_logprobs,
                                 const void *logits, int64_t logits_row_stride, int32_t logits_is_fp32,
                                 const float *temperatures, const int32_t *tokens, int32_t rows, int32_t vocab,
                                 int32_t top_k, pa_stream_t stream) {
    using namespace pa;
    if (rows < 0 || vocab < 0) return fail(PA_ERR_INVALID_ARG, "negative size");
    if (rows == 0) return PA_OK;
    if (vocab == 0) return fail(PA_ERR_INVALID_ARG, "vocab must be positive");
    if (vocab > 1 << 30) return fail(PA_ERR_UNSUPPORTED, "vocab %d (at most 2^30)", vocab);
    if (top_k < 0 || top_k > vocab) return fail(PA_ERR_INVALID_ARG, "top_k must be in [0, vocab]");
    if (top_k > LP_MAX_TOP) return fail(PA_ERR_UNSUPPORTED, "top_k %d (at most %d)", top_k, LP_MAX_TOP);
    if (!logprobs || !entropy || !logits || !tokens || (top_k > 0 && (!top_ids || !top_logprobs)))
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (logits_is_fp32 != 0 && logits_is_fp32 != 1) return fail(PA_ERR_INVALID_ARG, "logits_is_fp32 must be 0 or 1");
    const int align = logits_is_fp32 ? 4 : 8;  // elements per 16 bytes
    if (logits_row_stride < vocab || logits_row_stride % align)
        return fail(PA_ERR_INVALID_ARG, "logits_row_stride must be >= vocab and a multiple of %d", align);
    if (!aligned16(logits)) return fail(PA_ERR_INVALID_ARG, "logits must be 16-byte aligned");
    const int sms = sm_count();
    if (sms <= 0) return fail(PA_ERR_CUDA, "no CUDA device");
    LpArgs a = {};
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.logits = logits;
    a.stride = logits_row_stride;
    a.temperatures = temperatures;
    a.tokens = tokens;
    a.vocab = vocab;
    a.top = top_k;
    a.cluster = lp_ctas_per_row(rows, vocab, sms);
    a.err = device_error_ptr();
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (lp_threads((int64_t)rows * a.cluster, (vocab + a.cluster - 1) / a.cluster, sms) == 128)
        return logits_is_fp32 ? launch_logprobs<true, 128>(a, rows, s) : launch_logprobs<false, 128>(a, rows, s);
    return logits_is_fp32 ? launch_logprobs<true, 256>(a, rows, s) : launch_logprobs<false, 256>(a, rows, s);
}
