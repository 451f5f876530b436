// token_logprobs.cu -- log probabilities of given tokens, log-sum-exp, entropy and the
// largest alternatives of rows of logits, and their gradient (sm_103a).
//
// With s = scale x, m = max s, and Z = sum e^(s - m) = 1 + R (R: all but one largest):
//   lse = m + ln Z,   logp_v = s_v - m - ln Z,   H = ln Z - sum e^(s-m) (s - m) / Z
//   gradient   p_v = e^(s_v - lse),
//   dx_v = scale (dlogp (1[v = target] - p_v) - dH p_v (s_v - lse + H) + dlse p_v)
//
// Forward: one pass over a row, every thread with a running maximum and sums relative to
// it, joined over the block and, where rows are few, over a cluster of blocks that share a
// row.  The pass does nothing for the top k but keep each thread's maximum: the k-th
// largest of those bounds the k-th largest value from below, and only the threads at or
// above it, k of them but for ties, can hold one of the k; what they read is looked at
// once more (it is still in L2).  The gradient is one pass without any sum.
//
// What bounds them: HBM; the forward pass needs an exponential for every logit, 16 a clock
// and SM, where HBM delivers 11.8 logits of 16 bits.
#include <cooperative_groups.h>
#include <float.h>

#include "rn_common.cuh"
#include "rn_host.h"

namespace rn {

namespace cg = cooperative_groups;

static __device__ unsigned int g_logprobs_status = 0u;

// ---- element formats ----------------------------------------------------------------
// A row is read in granules of 16 bytes.  kLowBit: the lowest bit in which the ordered
// keys (below) of two values of the format can differ.

struct Row16Bf {
    using E = Bf16;
    using T = uint16_t;
    static constexpr int kElems = 8, kLowBit = 16;
    __device__ static __forceinline__ float one(T v) { return bf_lo(v); }
    __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
        return *reinterpret_cast<uint32_t *>(&r);
    }
};
struct Row16Half {
    using E = F16;
    using T = uint16_t;
    static constexpr int kElems = 8, kLowBit = 13;
    __device__ static __forceinline__ float one(T v) { return F16::lo(v); }
    __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        __half2 r = __hmax2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
        return *reinterpret_cast<uint32_t *>(&r);
    }
};
struct Row32 {
    using E = void;
    using T = float;
    static constexpr int kElems = 4, kLowBit = 0;
    __device__ static __forceinline__ float one(T v) { return v; }
};

template <class F>
__device__ __forceinline__ void widen(const uint4 &u, float (&x)[F::kElems]) {
    if constexpr (F::kElems == 8) {
        using E = typename F::E;
        x[0] = E::lo(u.x); x[1] = E::hi(u.x); x[2] = E::lo(u.y); x[3] = E::hi(u.y);
        x[4] = E::lo(u.z); x[5] = E::hi(u.z); x[6] = E::lo(u.w); x[7] = E::hi(u.w);
    } else {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
}
template <class F>
__device__ __forceinline__ uint4 narrow(const float (&x)[F::kElems]) {
    if constexpr (F::kElems == 8) {
        using E = typename F::E;
        return make_uint4(E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]), E::pack(x[6], x[7]));
    } else {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
}
template <class F>
__device__ __forceinline__ void store_one(typename F::T *p, float v) {
    if constexpr (F::kElems == 8)
        *p = static_cast<uint16_t>(F::E::pack(v, v));
    else
        *p = v;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest of a granule; NaN where it holds one.
template <class F>
__device__ __forceinline__ float largest(const uint4 &u) {
    if constexpr (F::kElems == 8) {
        const uint32_t w = F::max2(F::max2(u.x, u.y), F::max2(u.z, u.w));
        return max_nan(F::E::lo(w), F::E::hi(w));
    } else {
        return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                       max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
}

// 32 bits that are ordered as the values are, NaN above all; never 0, so 0 is "none".
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    if (key == 0xFFFFFFFFu) return __uint_as_float(0x7FFFFFFFu);
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// An entry of a list: larger for larger values, then for lower indices; 0 is "none".
__device__ __forceinline__ uint64_t entry(uint32_t key, int64_t index) {
    return static_cast<uint64_t>(key) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}

// 2^t to 2^-22 of it; zero below 2^-126.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---- a row --------------------------------------------------------------------------------
// Granules of a row lie on 16-byte boundaries; its first and last may begin before or end
// behind it, and only the elements that are the row's are read then.
template <class F>
struct Row {
    const typename F::T *x;
    int64_t V;
    int off;           // elements of the first granule in front of the row
    int64_t granules;

    __device__ __forceinline__ Row(const void *logits, int64_t stride, int64_t t, int64_t V_) : V(V_) {
        x = static_cast<const typename F::T *>(logits) + t * stride;
        off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(typename F::T));
        granules = (off + V + F::kElems - 1) / F::kElems;
    }
    // index of a granule's first element (that of the first may be negative)
    __device__ __forceinline__ int64_t index(int64_t g) const { return g * F::kElems - off; }
    __device__ __forceinline__ bool whole(int64_t g) const {
        const int64_t i = index(g);
        return i >= 0 && i + F::kElems <= V;
    }
    __device__ __forceinline__ uint4 load(int64_t g) const { return *reinterpret_cast<const uint4 *>(x + index(g)); }
    // A granule's elements, -infinity where it has none; a bit for each that there is.
    __device__ __forceinline__ uint32_t fetch(int64_t g, float (&v)[F::kElems]) const {
        const int64_t i = index(g);
        if (whole(g)) {
            widen<F>(load(g), v);
            return (1u << F::kElems) - 1u;
        }
        uint32_t there = 0u;
#pragma unroll
        for (int e = 0; e < F::kElems; ++e) {
            const bool in = i + e >= 0 && i + e < V;
            v[e] = in ? F::one(x[i + e]) : -INFINITY;
            there |= in ? 1u << e : 0u;
        }
        return there;
    }
};

// ---- forward ------------------------------------------------------------------------------

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowBatch = 4;      // granules a thread has under way
constexpr int kMostTop = 32;      // alternatives
constexpr int kMostCluster = 8;   // blocks of a row
constexpr int kFewThreads = 64;   // threads whose granules are looked at again one by one
constexpr int kList = 1024;       // entries of the list

struct LogprobsArgs {
    const void *logits;
    int64_t stride;
    const int64_t *targets;
    int64_t T, V;
    float scale, scale_log2;
    int k;
    int blocks;   // of a row: the cluster's
    float *logprobs, *lse, *entropy, *top_logprobs;
    int64_t *top_ids;
};

// A thread's running sums: m the largest so far, z = sum 2^t and s = sum 2^t t over its
// elements, t = (x - m) scale log2 e.  t stops at -200, where 2^t is zero: a product with
// the -infinity of a banned token would be NaN.  (A NaN leaves z and s as they are, and m
// says so; with m infinite all t stop there.)
struct Running {
    float m, z, s;

    __device__ __forceinline__ void raise(float to, float scale) {
        to = max_nan(to, m);  // (a NaN stays)
        const float t = fmaxf((m - to) * scale, -200.0f), f = exp2_fast(t);
        s = f * fmaf(t, z, s);
        z *= f;
        m = to;
    }
    __device__ __forceinline__ void add(float x, float scale) {
        const float t = fmaxf((x - m) * scale, -200.0f), e = exp2_fast(t);
        z += e;
        s = fmaf(e, t, s);
    }
};

struct RowShared {
    uint32_t keys[kRowWarps];
    float z[kRowWarps], s[kRowWarps];
    int owner;           // the lowest thread whose maximum is the block's
    float owner_z;
    // what the cluster's first block reads: the block's maximum, R and the sum of e t
    uint32_t max_key;
    float rest, sum_t;
    int cand[kFewThreads];
    int cands;
    int listed;          // entries wanted in the list (it holds kList)
    int counts[kRowWarps];
    uint64_t best[kRowWarps];
    uint64_t top[kMostTop];   // the block's largest, in order; 0 behind the last
    uint64_t list[kList];
};

template <class F>
__device__ __forceinline__ void push(RowShared &sh, const Row<F> &row, int64_t g, uint32_t least, bool above) {
    float v[F::kElems];
    const uint32_t there = row.fetch(g, v);
#pragma unroll
    for (int e = 0; e < F::kElems; ++e) {
        const uint32_t key = ordered(v[e]);
        if ((there >> e & 1u) && (above ? key > least : key >= least)) {
            const int at = atomicAdd(&sh.listed, 1);
            if (at < kList) sh.list[at] = entry(key, row.index(g) + e);
        }
    }
}

// The block's k largest of granules [g0, g1), thread i having read g0 + i, g0 + i +
// kRowThreads, ..; `key` its largest's, 0 where it read none.  Leaves them in sh.top.
template <class F>
__device__ void block_top(RowShared &sh, const Row<F> &row, int64_t g0, int64_t g1, uint32_t key, int k) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // least: the largest key that k threads reach (0: fewer than k read anything)
    uint32_t least = 0u;
    int reach = 0;
    for (int bit = 31; bit >= F::kLowBit; --bit) {
        // (below a negative value's lowest bit that differs its key is all ones)
        const uint32_t mid = least | 1u << bit;
        const int n = __syncthreads_count(key >= mid);
        if (n >= k) {
            least = mid;
            reach = n;
        }
    }
    if (least == 0u) reach = __syncthreads_count(key != 0u);
    if (tid == 0) sh.cands = sh.listed = 0;
    if (tid < kMostTop) sh.top[tid] = 0u;
    __syncthreads();
    // the least key of a value: the bits below kLowBit say nothing
    const uint32_t wanted = least == 0u ? 1u : least;
    const bool few = reach <= kFewThreads;
    // few threads reach it: theirs at least that large.  Else many values equal it: those
    // above it, of fewer than k threads, and then equal ones in the order of their indices.
    constexpr uint32_t kRest = (1u << F::kLowBit) - 1u;
    const bool mine = few ? key >= wanted : key > (least | kRest);
    if (mine) {
        const int at = atomicAdd(&sh.cands, 1);
        sh.cand[at] = tid;
    }
    __syncthreads();
    for (int i = warp; i < sh.cands; i += kRowWarps)
        for (int64_t g = g0 + sh.cand[i] + static_cast<int64_t>(lane) * kRowThreads; g < g1; g += 32ll * kRowThreads)
            push<F>(sh, row, g, few ? wanted : (least | kRest), !few);
    __syncthreads();
    if (!few && sh.listed < k) {
        int have = sh.listed;
        for (int64_t base = g0; base < g1 && have < k; base += kRowThreads) {
            float v[F::kElems];
            uint32_t equal = 0u;
            if (base + tid < g1) {
                const uint32_t there = row.fetch(base + tid, v);
#pragma unroll
                for (int e = 0; e < F::kElems; ++e)
                    if ((there >> e & 1u) && (ordered(v[e]) | kRest) == (least | kRest)) equal |= 1u << e;
            }
            int before = __popc(equal);
            const int n = before;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += w;
            }
            if (lane == 31) sh.counts[warp] = before;
            __syncthreads();
            int total = 0;
            before += have - n;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) {
                if (w < warp) before += sh.counts[w];
                total += sh.counts[w];
            }
#pragma unroll
            for (int e = 0; e < F::kElems; ++e)
                if (equal >> e & 1u) {
                    if (before < k) sh.list[before] = entry(ordered(v[e]), row.index(base + tid) + e);
                    ++before;
                }
            have += total;
            __syncthreads();
        }
        if (tid == 0) sh.listed = have < k ? have : k;
        __syncthreads();
    }
    const int n = sh.listed;
    if (n <= kList) {
        for (int i = tid; i < n; i += kRowThreads) {
            const uint64_t me = sh.list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += sh.list[j] > me ? 1 : 0;
            if (rank < k) sh.top[rank] = me;
        }
        __syncthreads();
        return;
    }
    // more than the list holds, all in few threads' granules: the largest below the last,
    // k times
    uint64_t last = ~0ull;
    for (int r = 0; r < k; ++r) {
        uint64_t best = 0u;
        for (int64_t g = g0 + tid; g < g1; g += kRowThreads) {
            float v[F::kElems];
            const uint32_t there = row.fetch(g, v);
#pragma unroll
            for (int e = 0; e < F::kElems; ++e) {
                const uint64_t c = there >> e & 1u ? entry(ordered(v[e]), row.index(g) + e) : 0u;
                if (c < last && c > best) best = c;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t w = __shfl_xor_sync(0xffffffffu, best, o);
            if (w > best) best = w;
        }
        if (lane == 0) sh.best[warp] = best;
        __syncthreads();
        for (int w = 0; w < kRowWarps; ++w)
            if (sh.best[w] > best) best = sh.best[w];
        if (tid == 0) sh.top[r] = best;
        last = best;
        __syncthreads();
    }
}

template <class F, bool CLUSTER>
__global__ void __launch_bounds__(kRowThreads, 2) logprobs_fwd_kernel(const __grid_constant__ LogprobsArgs a) {
    __shared__ RowShared sh;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x % a.blocks) : 0;
    const int64_t t = CLUSTER ? blockIdx.x / a.blocks : blockIdx.x;
    const Row<F> row(a.logits, a.stride, t, a.V);
    int64_t g0 = 0, g1 = row.granules;
    if (CLUSTER) {
        const int64_t per = (row.granules + a.blocks - 1) / a.blocks;
        g0 = per * rank < g1 ? per * rank : g1;
        g1 = g0 + per < g1 ? g0 + per : g1;
    }
    // the given token's logit comes while the row is read
    int64_t target = -1;
    float given = 0.0f;
    if (rank == 0 && tid == 0 && a.targets) {
        target = a.targets[t];
        if (target >= 0 && target < a.V) given = F::one(row.x[target]);
    }

    Running run = {-INFINITY, 0.0f, 0.0f};
    const float c = a.scale_log2;
    // granules that lie in the row as a whole
    const int64_t w1 = g1 > g0 && row.whole(g1 - 1) ? g1 : g1 - 1;
    int64_t g = g0 + tid;
    if (g < g1 && g == 0 && !row.whole(0)) g += kRowThreads;
    for (; g + (kRowBatch - 1) * kRowThreads < w1; g += kRowBatch * kRowThreads) {
        uint4 u[kRowBatch];
#pragma unroll
        for (int b = 0; b < kRowBatch; ++b) u[b] = row.load(g + b * kRowThreads);
        float m = largest<F>(u[0]);
#pragma unroll
        for (int b = 1; b < kRowBatch; ++b) m = max_nan(m, largest<F>(u[b]));
        if (!(m <= run.m)) run.raise(m, c);
#pragma unroll
        for (int b = 0; b < kRowBatch; ++b) {
            float v[F::kElems];
            widen<F>(u[b], v);
#pragma unroll
            for (int e = 0; e < F::kElems; ++e) run.add(v[e], c);
        }
    }
    for (; g < w1; g += kRowThreads) {
        const uint4 u = row.load(g);
        const float m = largest<F>(u);
        if (!(m <= run.m)) run.raise(m, c);
        float v[F::kElems];
        widen<F>(u, v);
#pragma unroll
        for (int e = 0; e < F::kElems; ++e) run.add(v[e], c);
    }
    // the row's ends, by the threads whose turn it would be
    const auto part = [&](int64_t at) {
        float v[F::kElems];
        row.fetch(at, v);
        for (int e = 0; e < F::kElems; ++e) {
            if (!(v[e] <= run.m)) run.raise(v[e], c);
            run.add(v[e], c);
        }
    };
    if (g1 > g0) {
        if (g0 == 0 && tid == 0 && !row.whole(0)) part(0);
        const int64_t last = g1 - 1;
        if (last != 0 && !row.whole(last) && (last - g0) % kRowThreads == tid) part(last);
    }

    // the block's maximum and sums
    const uint32_t key = g0 + tid < g1 ? ordered(run.m) : 0u;
    const uint32_t warp_key = __reduce_max_sync(0xffffffffu, key);
    if (lane == 0) sh.keys[warp] = warp_key;
    if (tid == 0) sh.owner = kRowThreads;
    __syncthreads();
    uint32_t top_key = 0u;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) top_key = max(top_key, sh.keys[w]);
    // a thread with the maximum counts apart: its sum is 1 and what may be little beside it
    if (key == top_key && key != 0u) atomicMin(&sh.owner, tid);
    __syncthreads();
    const float m = top_key == 0u ? -INFINITY : value_of(top_key);
    {
        const float shift = fmaxf((run.m - m) * c, -200.0f), f = exp2_fast(shift);
        float z = f * run.z, s = f * fmaf(shift, run.z, run.s);
        if (tid == sh.owner) {
            sh.owner_z = z;
            z = 0.0f;
        }
        z = warp_sum(z);
        s = warp_sum(s);
        if (lane == 0) {
            sh.z[warp] = z;
            sh.s[warp] = s;
        }
    }
    __syncthreads();
    float rest = 0.0f, sum_t = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
        rest += sh.z[w];
        sum_t += sh.s[w];
    }
    if (sh.owner < kRowThreads) {
        if (rest + sh.owner_z >= 2.0f) {
            rest += sh.owner_z - 1.0f;
        } else if (warp == 0) {
            // one token holds more than half of the sum: the owner's others once more, alone
            float r = 0.0f;
            for (int64_t at = g0 + sh.owner + static_cast<int64_t>(lane) * kRowThreads; at < g1;
                 at += 32ll * kRowThreads) {
                float v[F::kElems];
                row.fetch(at, v);
#pragma unroll
                for (int e = 0; e < F::kElems; ++e)
                    if (v[e] < m) r += exp2_fast(fmaxf((v[e] - m) * c, -200.0f));
            }
            rest += warp_sum(r);
        }
    }
    // (warp 0's are complete)
    if (tid == 0) {
        sh.max_key = top_key;
        sh.rest = rest;
        sh.sum_t = sum_t;
    }

    if (a.k > 0) block_top<F>(sh, row, g0, g1, key, a.k);

    float row_m = m, row_rest = rest, row_t = sum_t;
    if constexpr (CLUSTER) {
        auto cluster = cg::this_cluster();
        cluster.sync();
        if (rank == 0) {
            // joins the blocks' sums in their order
            const int n = a.blocks;
            uint32_t most = 0u;
            for (int b = 0; b < n; ++b) most = max(most, *cluster.map_shared_rank(&sh.max_key, b));
            row_m = value_of(most);
            row_rest = row_t = 0.0f;
            bool found = false;
            for (int b = 0; b < n; ++b) {
                const uint32_t bk = *cluster.map_shared_rank(&sh.max_key, b);
                if (bk == 0u) continue;
                const float br = *cluster.map_shared_rank(&sh.rest, b), bt = *cluster.map_shared_rank(&sh.sum_t, b);
                const float shift = fmaxf((value_of(bk) - row_m) * c, -200.0f), f = exp2_fast(shift);
                row_t += f * fmaf(shift, 1.0f + br, bt);
                if (bk == most && !found) {
                    found = true;
                    row_rest += br;
                } else {
                    row_rest += f * (1.0f + br);
                }
            }
            if (a.k > 0) {
                // ranks the blocks' entries; equal ones are no entries
                uint64_t me = 0u;
                if (tid < n * kMostTop) me = *cluster.map_shared_rank(&sh.top[tid % kMostTop], tid / kMostTop);
                if (tid < n * kMostTop) sh.list[tid] = me;
                __syncthreads();
                int r = 0;
                if (me != 0u)
                    for (int j = 0; j < n * kMostTop; ++j) r += sh.list[j] > me ? 1 : 0;
                __syncthreads();
                if (me != 0u && r < a.k) sh.list[kList - kMostTop + r] = me;
                __syncthreads();
                if (tid < a.k) sh.top[tid] = sh.list[kList - kMostTop + tid];
                __syncthreads();
            }
        }
        cluster.sync();  // the others' shared memory is read until here
        if (rank != 0) return;
    }
    // rank 0, every thread of it with the row's maximum and warp 0 with its sums
    const bool plain = row_m > -INFINITY && row_m < INFINITY;
    if (warp == 0) {
        const float z = 1.0f + row_rest, ln_z = log1pf(row_rest);
        const float none = row_m == -INFINITY ? 0.0f : __uint_as_float(0x7FFFFFFFu);
        const float entropy = plain ? fmaf(-0.6931471805599453f, row_t / z, ln_z) : none;
        const auto logp = [&](float x) {
            if (plain) return (x - row_m) * a.scale - ln_z;
            if (row_m == -INFINITY) return -INFINITY;
            return x == INFINITY || !(row_m == row_m) ? __uint_as_float(0x7FFFFFFFu) : x - row_m;
        };
        if (lane == 0) {
            if (a.lse) a.lse[t] = plain ? fmaf(row_m, a.scale, ln_z) : row_m;
            if (a.entropy) a.entropy[t] = entropy;
            if (a.logprobs) {
                float v = 0.0f;
                if (target >= a.V) {
                    atomicOr(&g_logprobs_status, RN_STATUS_BAD_INDEX);
                    v = __uint_as_float(0x7FFFFFFFu);
                } else if (target >= 0) {
                    v = logp(given);
                }
                a.logprobs[t] = v;
            }
        }
        if (lane < a.k) {
            const uint64_t e = sh.top[lane];
            a.top_logprobs[t * a.k + lane] = logp(value_of(static_cast<uint32_t>(e >> 32)));
            a.top_ids[t * a.k + lane] = 0xFFFFFFFFu - static_cast<uint32_t>(e);
        }
    }
}

// ---- gradient --------------------------------------------------------------------------------

struct LogprobsGradArgs {
    const void *logits;
    int64_t stride;
    const int64_t *targets;
    const float *logprobs, *lse, *entropy;
    const float *dlogprobs, *dentropy, *dlse;
    int64_t dlogprobs_stride, dentropy_stride, dlse_stride;
    int64_t T, V;
    float scale;
    void *dlogits;
    int64_t dstride;
    int64_t chunks;  // blocks of a row
};

constexpr int kGradThreads = 256;
constexpr int kGradBatch = 4;  // granules of a thread

template <class F>
__global__ void __launch_bounds__(kGradThreads) logprobs_bwd_kernel(const __grid_constant__ LogprobsGradArgs a) {
    pdl_trigger();
    pdl_wait();
    const int64_t t = blockIdx.x / a.chunks, chunk = blockIdx.x - t * a.chunks;
    const Row<F> row(a.logits, a.stride, t, a.V);
    typename F::T *out = static_cast<typename F::T *>(a.dlogits) + t * a.dstride;
    const bool aligned = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.x)) & 15u) == 0;
    const int64_t first = chunk * (kGradThreads * kGradBatch) + threadIdx.x;
    uint4 u[kGradBatch];
#pragma unroll
    for (int b = 0; b < kGradBatch; ++b) {
        const int64_t g = first + b * kGradThreads;
        u[b] = make_uint4(0u, 0u, 0u, 0u);
        if (g < row.granules && row.whole(g)) u[b] = row.load(g);
    }
    const float lse = a.lse[t];
    const float h = a.entropy ? a.entropy[t] : 0.0f;
    const float dh = a.dentropy ? a.dentropy[t * a.dentropy_stride] : 0.0f;
    const float dl = a.dlse ? a.dlse[t * a.dlse_stride] : 0.0f;
    int64_t target = -1;
    float dp = 0.0f, lt = 0.0f;
    if (a.dlogprobs) {
        target = a.targets[t];
        if (target >= 0) {
            dp = a.dlogprobs[t * a.dlogprobs_stride];
            lt = a.logprobs[t];
        }
    }
    // dx = p (c0 - c1 (s - lse)); s - lse stops at -150, where p is zero and a product with
    // the -infinity of a banned token would be NaN
    float c0 = a.scale * (dl - dp - dh * h);
    const float c1 = a.scale * dh;
    const float nan = __uint_as_float(0x7FFFFFFFu);
    if (!(lse < INFINITY)) c0 = nan;  // NaN or +infinity
    if (target >= a.V) {
        c0 = nan;
        if (chunk == 0 && threadIdx.x == 0) atomicOr(&g_logprobs_status, RN_STATUS_BAD_INDEX);
    }
    // of the given token, by its own log probability: 1 - p where p is nearly 1
    const auto given = [&] {
        if (!(lse < INFINITY)) return nan;
        if (lse == -INFINITY) return 0.0f;
        const float l = fmaxf(lt, -150.0f);
        return a.scale * (expf(l) * (dl - dh * (l + h)) - expm1f(l) * dp);
    };
    const auto grad = [&](float x) {
        const float l = fmaxf(fmaf(x, a.scale, -lse), -150.0f);
        return exp2_fast(l * 1.4426950408889634f) * fmaf(-c1, l, c0);
    };
#pragma unroll
    for (int b = 0; b < kGradBatch; ++b) {
        const int64_t g = first + b * kGradThreads;
        if (g >= row.granules) return;
        const int64_t i = row.index(g);
        float v[F::kElems];
        uint32_t there = (1u << F::kElems) - 1u;
        const bool whole = row.whole(g);
        if (whole)
            widen<F>(u[b], v);
        else
            there = row.fetch(g, v);
#pragma unroll
        for (int e = 0; e < F::kElems; ++e) v[e] = grad(v[e]);
        if (target >= i && target < i + F::kElems) {
            const float gt = given();
#pragma unroll
            for (int e = 0; e < F::kElems; ++e)
                if (target == i + e) v[e] = gt;
        }
        if (whole && aligned) {
            st16(out + i, narrow<F>(v));
        } else {
#pragma unroll
            for (int e = 0; e < F::kElems; ++e)
                if (there >> e & 1u) store_one<F>(out + i + e, v[e]);
        }
    }
}

// ---- host ---------------------------------------------------------------------------------------

static int elem_bytes(int dtype) { return dtype == RN_DTYPE_F32 ? 4 : 2; }

// Blocks that share a row: more where rows are too few to fill the GPU.
static int row_blocks(int64_t T, int64_t V, int dtype, int sm_count) {
    int n = 1;
    const int64_t granules = V * elem_bytes(dtype) / 16;
    while (n < kMostCluster && T * n < 4 * static_cast<int64_t>(sm_count) && granules / (2 * n) >= kRowThreads) n *= 2;
    return n;
}

template <class F, bool CLUSTER>
static int launch_fwd(const LogprobsArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.T * a.blocks));
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.blocks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, logprobs_fwd_kernel<F, CLUSTER>, a) != cudaSuccess) {
        cudaGetLastError();
        return RN_ERR_LAUNCH;
    }
    return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_LAUNCH;
}

template <class F>
static int run_fwd(const LogprobsArgs &a, cudaStream_t st) {
    return a.blocks > 1 ? launch_fwd<F, true>(a, st) : launch_fwd<F, false>(a, st);
}

template <class F>
static int run_bwd(const LogprobsGradArgs &a, cudaStream_t st) {
    return launch_pdl(logprobs_bwd_kernel<F>, dim3(static_cast<unsigned>(a.T * a.chunks)), dim3(kGradThreads), 0, st,
                      a);
}

// What both calls check of their logits.
static int check_rows(int dtype, int64_t stride, int64_t T, int64_t V, float scale) {
    if (dtype != RN_DTYPE_BF16 && dtype != RN_DTYPE_F16 && dtype != RN_DTYPE_F32) return RN_ERR_ARG;
    if (T < 0 || T > (INT32_MAX >> 3) || V < 1 || V > INT32_MAX - 64) return RN_ERR_SHAPE;
    if (T > 1 && stride < V) return RN_ERR_SHAPE;
    if (!(scale > 0.0f) || !(scale <= FLT_MAX / 2)) return RN_ERR_ARG;
    return RN_OK;
}
static bool misaligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

int logprobs_status(unsigned int *out, int clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_logprobs_status, sizeof v) != cudaSuccess) {
        cudaGetLastError();
        return RN_ERR_DEVICE;
    }
    if (clear && v != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_logprobs_status, &zero, sizeof zero) != cudaSuccess) {
            cudaGetLastError();
            return RN_ERR_DEVICE;
        }
    }
    *out = v;
    return RN_OK;
}

}  // namespace rn

extern "C" {

int token_logprobs_fwd(int dtype, const void *logits, int64_t stride, const int64_t *targets, int64_t T, int64_t V,
                       float scale, int top_k, float *logprobs, float *lse, float *entropy, float *top_logprobs,
                       int64_t *top_ids, rn_stream_t stream) {
    int rc = rn::check_rows(dtype, stride, T, V, scale);
    if (rc != RN_OK) return rc;
    if (top_k < 0 || top_k > rn::kMostTop || top_k > V) return RN_ERR_SHAPE;
    if (T == 0) return RN_OK;
    if (!logits || (logprobs && !targets) || (top_k > 0 && (!top_logprobs || !top_ids))) return RN_ERR_NULL;
    if (rn::misaligned(logits, rn::elem_bytes(dtype)) || rn::misaligned(targets, 8) || rn::misaligned(logprobs, 4) ||
        rn::misaligned(lse, 4) || rn::misaligned(entropy, 4) || rn::misaligned(top_logprobs, 4) ||
        rn::misaligned(top_ids, 8))
        return RN_ERR_ALIGN;
    const rn::DeviceInfo *dev = rn::current_device_info();
    if (!dev) return RN_ERR_DEVICE;
    rn::LogprobsArgs a = {};
    a.logits = logits;
    a.stride = stride;
    a.targets = logprobs ? targets : nullptr;
    a.T = T;
    a.V = V;
    a.scale = scale;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.k = top_k;
    a.blocks = rn::row_blocks(T, V, dtype, dev->sm_count);
    a.logprobs = logprobs;
    a.lse = lse;
    a.entropy = entropy;
    a.top_logprobs = top_logprobs;
    a.top_ids = top_ids;
    const auto st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == RN_DTYPE_F32) return rn::run_fwd<rn::Row32>(a, st);
    if (dtype == RN_DTYPE_F16) return rn::run_fwd<rn::Row16Half>(a, st);
    return rn::run_fwd<rn::Row16Bf>(a, st);
}

int token_logprobs_bwd(int dtype, const void *logits, int64_t stride, const int64_t *targets, const float *logprobs,
                       const float *lse, const float *entropy, const float *dlogprobs, int64_t dlogprobs_stride,
                       const float *dentropy, int64_t dentropy_stride, const float *dlse, int64_t dlse_stride,
                       int64_t T, int64_t V, float scale, void *dlogits, int64_t dlogits_stride, rn_stream_t stream) {
    int rc = rn::check_rows(dtype, stride, T, V, scale);
    if (rc != RN_OK) return rc;
    if (T > 1 && dlogits_stride < V) return RN_ERR_SHAPE;
    if (dlogprobs_stride < 0 || dentropy_stride < 0 || dlse_stride < 0) return RN_ERR_SHAPE;
    if (T == 0) return RN_OK;
    if (!logits || !lse || !dlogits || (dlogprobs && (!targets || !logprobs)) || (dentropy && !entropy))
        return RN_ERR_NULL;
    const int bytes = rn::elem_bytes(dtype);
    if (rn::misaligned(logits, bytes) || rn::misaligned(dlogits, bytes) || rn::misaligned(targets, 8) ||
        rn::misaligned(logprobs, 4) || rn::misaligned(lse, 4) || rn::misaligned(entropy, 4) ||
        rn::misaligned(dlogprobs, 4) || rn::misaligned(dentropy, 4) || rn::misaligned(dlse, 4))
        return RN_ERR_ALIGN;
    const int64_t elems = 16 / bytes, per = static_cast<int64_t>(rn::kGradThreads) * rn::kGradBatch;
    rn::LogprobsGradArgs a = {};
    // (a row that begins inside a granule may touch one more)
    const bool inside = rn::misaligned(logits, 16) || (T > 1 && stride * bytes % 16 != 0);
    a.chunks = ((V + elems - 1) / elems + (inside ? 1 : 0) + per - 1) / per;
    if (a.chunks > INT32_MAX / T) return RN_ERR_SHAPE;
    a.logits = logits;
    a.stride = stride;
    a.targets = targets;
    a.logprobs = logprobs;
    a.lse = lse;
    a.entropy = dentropy ? entropy : nullptr;
    a.dlogprobs = dlogprobs;
    a.dlogprobs_stride = dlogprobs_stride;
    a.dentropy = dentropy;
    a.dentropy_stride = dentropy_stride;
    a.dlse = dlse;
    a.dlse_stride = dlse_stride;
    a.T = T;
    a.V = V;
    a.scale = scale;
    a.dlogits = dlogits;
    a.dstride = dlogits_stride;
    const auto st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == RN_DTYPE_F32) return rn::run_bwd<rn::Row32>(a, st);
    if (dtype == RN_DTYPE_F16) return rn::run_bwd<rn::Row16Half>(a, st);
    return rn::run_bwd<rn::Row16Bf>(a, st);
}

}  // extern "C"
