// token_logprobs.cu -- log probabilities of given tokens, log-sum-exp, entropy and the
// largest alternatives of rows of logits, and their gradient (sm_103a).
//
// With s = scale x, m = max s, and Z = sum e^(s - m) = 1 + R (R: all but one largest):
//   lse = m + ln Z,   logp_v = s_v - m - ln Z,   H = ln Z - sum e^(s-m) (s - m) / Z
//   gradient   p_v = e^(s_v - lse),
//   dx_v = scale (dlogp (1[v = target] - p_v) - dH p_v (s_v - lse + H) + dlse p_v)
//
// Forward: one pass over a row, every thread with a running maximum and sums relative to a
// reference, joined over the block and, where rows are few, over a cluster of blocks that
// share a row.  The pass does nothing for the top k but note each thread's largest values of
// runs of its elements: the k-th largest of 32 groups of threads' bounds the k-th largest
// element from below, and only runs that reach it, little more than k of them but for ties,
// can hold one of the k; they are looked at once more (they are still in L2).  The gradient
// is one pass without any sum.
//
// What bounds the forward pass: HBM, with the issue slots not far behind.  A logit of 16 bits
// takes 6.3 instructions (one exponential, half each of a maximum, a clamp and three fused
// operations, one to widen it); with 8 alternatives the issue slots are 55% full at 1024 rows of
// 131072, the special function unit 30%.  2048 rows of 131072 normal logits in bf16: 83.5 us
// without alternatives, 6.43 TB/s, 86.9 with 8, 94.6 with 20 (to join a row takes a block, beside
// others that read, about 3500 clocks, 10000 and 16000).
#include <cooperative_groups.h>
#include <float.h>

#include <type_traits>

#include "rn_common.cuh"
#include "rn_host.h"

namespace rn {

namespace cg = cooperative_groups;

static __device__ unsigned int g_logprobs_status = 0u;

// ---- element formats ----------------------------------------------------------------
// A row is read in granules of 16 bytes.

struct Row16Bf {
    using E = Bf16;
    using T = uint16_t;
    static constexpr int kElems = 8;
    static constexpr uint32_t kNone = 0xFF80FF80u;  // a word of -infinity
    __device__ static __forceinline__ float one(T v) { return bf_lo(v); }
    __device__ static __forceinline__ uint32_t below2(float x) {  // two of the next value not above x
        return 0x10001u * __bfloat16_as_ushort(__float2bfloat16_rd(x));
    }
    __device__ static __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
        __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
        return *reinterpret_cast<uint32_t *>(&r);
    }
    __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
        return *reinterpret_cast<uint32_t *>(&r);
    }
};
struct Row16Half {
    using E = F16;
    using T = uint16_t;
    static constexpr int kElems = 8;
    static constexpr uint32_t kNone = 0xFC00FC00u;
    __device__ static __forceinline__ float one(T v) { return F16::lo(v); }
    __device__ static __forceinline__ uint32_t below2(float x) { return 0x10001u * __half_as_ushort(__float2half_rd(x)); }
    __device__ static __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
        __half2 r = __hmax2_nan(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
        return *reinterpret_cast<uint32_t *>(&r);
    }
    __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        __half2 r = __hmax2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
        return *reinterpret_cast<uint32_t *>(&r);
    }
};
struct Row32 {
    using E = void;
    using T = float;
    static constexpr int kElems = 4;
    static constexpr uint32_t kNone = 0xFF800000u;
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

// The largest of some granules; NaN where they hold one.
template <class F, int N>
__device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    if constexpr (F::kElems == 8) {
        uint32_t w = F::max2_nan(F::max2_nan(u[0].x, u[0].y), F::max2_nan(u[0].z, u[0].w));
#pragma unroll
        for (int i = 1; i < N; ++i)
            w = F::max2_nan(w, F::max2_nan(F::max2_nan(u[i].x, u[i].y), F::max2_nan(u[i].z, u[i].w)));
        return max_nan(F::E::lo(w), F::E::hi(w));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i)
            m = max_nan(m, max_nan(max_nan(__uint_as_float(u[i].x), __uint_as_float(u[i].y)),
                                   max_nan(__uint_as_float(u[i].z), __uint_as_float(u[i].w))));
        return m;
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

// Elements i .. of a row that are in [0, V), as a granule.  (A call: it would be in many places.)
template <class F>
__device__ __noinline__ uint4 end_of_row(const typename F::T *x, int i, int V) {
    uint32_t w[4] = {F::kNone, F::kNone, F::kNone, F::kNone};
#pragma unroll
    for (int e = 0; e < F::kElems; ++e)
        if (i + e >= 0 && i + e < V) {
            if constexpr (F::kElems == 8)
                w[e / 2] = __byte_perm(w[e / 2], x[i + e], e & 1 ? 0x5410 : 0x3254);
            else
                w[e] = __float_as_uint(x[i + e]);
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Granules of a row lie on 16-byte boundaries; its first and last may begin before or end
// behind it, and only the elements that are the row's are read then.
template <class F>
struct Row {
    const typename F::T *x;
    int V;
    int off;       // elements of the first granule in front of the row
    int granules;

    __device__ __forceinline__ Row(const void *logits, int64_t stride, int64_t t, int64_t V_) : V(static_cast<int>(V_)) {
        x = static_cast<const typename F::T *>(logits) + t * stride;
        off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(typename F::T));
        granules = (off + V + F::kElems - 1) / F::kElems;
    }
    // index of a granule's first element (that of the first may be negative)
    __device__ __forceinline__ int index(int g) const { return g * F::kElems - off; }
    __device__ __forceinline__ bool whole(int g) const {
        const int i = index(g);
        return i >= 0 && i <= V - F::kElems;
    }
    __device__ __forceinline__ uint4 load(int g) const { return *reinterpret_cast<const uint4 *>(x + index(g)); }
    // A granule, -infinity where it has no element.
    __device__ __forceinline__ uint4 fetch(int g) const { return whole(g) ? load(g) : end_of_row<F>(x, index(g), V); }
    // A bit for each element that a granule has.
    __device__ __forceinline__ uint32_t there(int g) const {
        const int i = index(g), lo = i < 0 ? -i : 0, hi = V - i < F::kElems ? V - i : F::kElems;
        return (1u << hi) - (1u << lo);
    }
};

// Element e of a granule.
template <class F>
__device__ __forceinline__ float element(const uint4 &u, int e) {
    const int word = F::kElems == 8 ? e >> 1 : e;
    const uint32_t w = word & 2 ? (word & 1 ? u.w : u.z) : (word & 1 ? u.y : u.x);
    if constexpr (F::kElems == 8)
        return e & 1 ? F::E::hi(w) : F::E::lo(w);
    else
        return __uint_as_float(w);
}

// ---- forward ------------------------------------------------------------------------------

// Batches that a thread has under way or is taking: as shared memory allows.
template <int NT>
constexpr int kStages = NT == 128 ? 3 : 2;
constexpr int kRowBatch = 4;      // granules of a batch
constexpr int kMostTop = 32;      // alternatives
// Blocks of an SM, by registers: 72 a thread in blocks of 64 and 128, 64 in the others.
constexpr int resident_blocks(int threads) { return (threads == 64 || threads == 128 ? 896 : 1024) / threads; }
constexpr int kMostCluster = 8;   // blocks of a row
constexpr int kList = 190;        // entries of the list
constexpr int kItems = 128;       // runs of batches that are looked at again
// The most runs of batches whose largest values a thread notes: as shared memory allows.
template <class F, int NT>
constexpr int kRuns = (NT == 64 ? 32 : NT == 128 ? 8 : 16) * F::kElems / 8;  // up to 32: bits of a word

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

// A thread's running sums: top the largest so far, z = sum 2^t and s = sum 2^t t over its
// elements, t = c x - r with c = scale log2 e and a reference r near c top.  Which number r is
// does not matter (nor its rounding), and it stays until c top passes it by kRoom: nearly
// always the first batch's largest does for the whole row.
constexpr float kRoom = 8.0f;
// t stops where 2^t is zero, at -200 or so: a product with the -infinity of a banned token
// would be NaN.  In 16 bits that is done two elements an instruction, on x, with the
// format's next value below; where there is none the thread's sums wait (shallow) for a
// second pass over its elements.  In 32 bits it is done on t.
constexpr float kDeep = 200.0f;
// References beyond this stand too far from c top for a power of two: the second pass, too.
constexpr float kFar = 0x1p20f;

template <class F>
struct Running {
    float top, r;
    float limit;      // the largest x that the reference serves
    uint32_t least;   // 16 bits: two of an x whose 2^t is zero; smaller ones count as it
    Pair z, s;
    bool shallow;     // there is no such x, or r is too far from c top

    // (The sums of what comes before the first finite x do not matter.)
    __device__ __forceinline__ Running()
        : top(-INFINITY), r(0.0f), limit(-INFINITY), least(0u), z(Pair::of(0.0f, 0.0f)), s(z), shallow(false) {}

    // (An infinity or NaN decides the row, and no sum matters.)
    __device__ __forceinline__ void refer(float to, float c) {
        if (!(fabsf(to) < INFINITY)) return;
        const float now = c * to;
        if (limit == -INFINITY) {
            z = s = Pair::of(0.0f, 0.0f);
        } else {
            const float t = fmaxf(r - now, -kDeep), f = exp2_fast(t);
            const Pair ff = Pair::of(f, f);
            s = ff * Pair::of(t, t).fma(z, s);
            z = ff * z;
        }
        r = now;
        limit = to + kRoom / c;
        if constexpr (F::kElems == 8) {
            least = F::below2(__fsub_rd(to, kDeep / c));
            shallow |= !(F::E::lo(least) > -INFINITY);
        }
        shallow |= !(fabsf(now) <= kFar);
    }
    __device__ __forceinline__ void add(Pair t) {
        const float2 x = t.split();
        const Pair e = Pair::of(exp2_fast(x.x), exp2_fast(x.y));
        z = z + e;
        s = e.fma(t, s);
    }
    // Adds N granules, the largest of them `most`.
    template <int N>
    __device__ __forceinline__ void take(const uint4 (&u)[N], float most, float c) {
        top = max_nan(top, most);
        if (!(most <= limit)) refer(most, c);
        const Pair cc = Pair::of(c, c), rr = Pair::of(-r, -r);
        if constexpr (F::kElems == 8) {
            const auto word = [&](uint32_t w) {
                w = F::max2(w, least);
                add(Pair::of(F::E::lo(w), F::E::hi(w)).fma(cc, rr));
            };
#pragma unroll
            for (int i = 0; i < N; ++i) {
                word(u[i].x);
                word(u[i].y);
                word(u[i].z);
                word(u[i].w);
            }
        } else {
            const auto two = [&](uint32_t a, uint32_t b) {
                const float2 t = Pair::of(__uint_as_float(a), __uint_as_float(b)).fma(cc, rr).split();
                add(Pair::of(fmaxf(t.x, -kDeep), fmaxf(t.y, -kDeep)));
            };
#pragma unroll
            for (int i = 0; i < N; ++i) {
                two(u[i].x, u[i].y);
                two(u[i].z, u[i].w);
            }
        }
    }
};

// A block's share of a row: granules g0 .. g1 - 1, of which w0 .. w1 - 1 lie in the row as a
// whole.  Thread i takes w0 + i, w0 + i + NT, ..; thread 0 the row's first granule as well
// if that is the block's and not whole, thread 1 the last.
struct Share {
    int g0, w0, w1, g1;

    template <class F>
    __device__ __forceinline__ Share(const Row<F> &row, int first, int end)
        : g0(first), w0(first < end && !row.whole(first) ? first + 1 : first), w1(end), g1(end) {
        if (w0 < end && !row.whole(end - 1)) --w1;
    }
    // what block `rank` of `blocks` has of a row
    template <class F>
    __device__ __forceinline__ static Share of(const Row<F> &row, int rank, int blocks) {
        const int per = (row.granules + blocks - 1) / blocks;
        const int64_t start = static_cast<int64_t>(per) * rank;
        const int g0 = start < row.granules ? static_cast<int>(start) : row.granules;
        return Share(row, g0, row.granules - g0 > per ? g0 + per : row.granules);
    }
    // the end of the row that a thread takes, or -1
    __device__ __forceinline__ int end_of(int tid) const {
        return tid == 0 && g0 < w0 ? g0 : (tid == 1 && w1 < g1 ? w1 : -1);
    }
};

// The sums of a thread's elements once more, by `top`, their largest, with t stopped by itself.
template <class F, int NT>
__device__ __noinline__ float2 sums_again(const void *x, int64_t V, float top, Share share, float c) {
    const Row<F> row(x, 0, 0, V);
    float z = 0.0f, s = 0.0f;
    const auto take = [&](int g) {
        const uint4 u = row.fetch(g);
#pragma unroll 1
        for (int e = 0; e < F::kElems; ++e) {
            const float t = fmaxf((element<F>(u, e) - top) * c, -kDeep), p = exp2_fast(t);
            z += p;
            s = fmaf(p, t, s);
        }
    };
    if (fabsf(top) < INFINITY) {
        for (int g = share.w0 + threadIdx.x; g < share.w1; g += NT) take(g);
        if (share.end_of(threadIdx.x) >= 0) take(share.end_of(threadIdx.x));
    }
    return make_float2(z, s);
}

// What one block of a row knows of it: its largest key (0: no element), what the sum of
// 2^t has beside one of the largest, and the sum of 2^t t, t by that largest.
struct RowPart {
    uint32_t key;
    float rest, sum_t;
};

// What a cluster's first block is told by all of them, of one row and the next.
struct ClusterShared {
    RowPart parts[2][kMostCluster];
    uint64_t tops[2][kMostCluster][kMostTop];
};
struct NoCluster {};

template <class F, int NT, bool CLUSTER>
struct RowShared {
    uint4 stage[kStages<NT>][kRowBatch][NT];    // batches under way, each thread's own
    alignas(16) uint64_t list[kList + 2];
    alignas(16) uint32_t groups[NT / 32][32];
    uint64_t best[NT / 32];
    uint64_t top[kMostTop];                     // the block's largest, in order; 0 behind the last
    uint32_t keys[NT];
    float z[NT / 32], s[NT / 32];
    float owner_z, owner_s;
    int listed;                                 // entries wanted in the list (it holds kList)
    int items;                                  // runs wanted in `item` (it holds kItems)
    int counts[NT / 32];
    float ends[2];                              // the largest of the row's ends
    int item[kItems];                           // thread and run
    typename F::T slots[kRuns<F, NT>][NT];      // by run of batches and thread: its largest
    std::conditional_t<CLUSTER, ClusterShared, NoCluster> cluster;
};

// Lists the elements of a granule that are no less than `least` (above: that are larger).
// (By floats, a NaN is listed whatever `least` is, and it ranks first.)
template <class F, class S>
__device__ __forceinline__ void push(S &sh, const Row<F> &row, int g, uint32_t least, bool above) {
    const uint4 u = row.fetch(g);
    float v[F::kElems];
    widen<F>(u, v);
    uint32_t hit = row.there(g);
    const float low = value_of(least);
#pragma unroll
    for (int e = 0; e < F::kElems; ++e)
        if (above ? v[e] <= low : v[e] < low) hit &= ~(1u << e);
    if (hit == 0u) return;
    int at = atomicAdd(&sh.listed, __popc(hit));
#pragma unroll 1
    for (; hit; hit &= hit - 1, ++at) {
        const int e = __ffs(hit) - 1;
        if (at < kList) sh.list[at] = entry(ordered(element<F>(u, e)), row.index(g) + e);
    }
}

// The granules of the threads of `lanes` of this warp, by the warp together.
template <class F, int NT, class S>
__device__ __forceinline__ void push_threads(S &sh, const Row<F> &row, const Share &share, uint32_t lanes,
                                             uint32_t least, bool above) {
    const int lane = threadIdx.x & 31, first = threadIdx.x - lane;
    while (lanes) {
        const int who = first + __ffs(lanes) - 1;
        lanes &= lanes - 1;
        for (int g = share.w0 + who + lane * NT; g < share.w1; g += 32 * NT) push<F>(sh, row, g, least, above);
        if (lane == 0 && share.end_of(who) >= 0) push<F>(sh, row, share.end_of(who), least, above);
    }
}

// Many elements equal `least`, or the list is full: lists those above it and, where these
// are fewer than k, equal ones in the order of their indices.  For all threads; sh.listed is
// what the list then needs to hold.
template <class F, int NT, class S>
__device__ __noinline__ void list_many(S &sh, const Row<F> &row, const Share &share, uint32_t key,
                                       uint32_t least, int k) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __syncthreads();
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    push_threads<F, NT>(sh, row, share, __ballot_sync(0xffffffffu, key > least), least, true);
    __syncthreads();
    int have = sh.listed;
    __syncthreads();
    if (have >= k) return;
    for (int base = share.g0; base < share.g1 && have < k; base += NT) {
        uint32_t equal = 0u;
        if (base + tid < share.g1) {
            float v[F::kElems];
            widen<F>(row.fetch(base + tid), v);
            const uint32_t there = row.there(base + tid);
#pragma unroll
            for (int e = 0; e < F::kElems; ++e)
                if ((there >> e & 1u) && ordered(v[e]) == least) equal |= 1u << e;
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
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) before += sh.counts[w];
            total += sh.counts[w];
        }
#pragma unroll
        for (int e = 0; e < F::kElems; ++e)
            if (equal >> e & 1u) {
                if (before < k) sh.list[before] = entry(least, row.index(base + tid) + e);
                ++before;
            }
        have += total;
        __syncthreads();
    }
    if (tid == 0) sh.listed = have < k ? have : k;
    __syncthreads();
}

// More elements above some value than the list holds, all in few threads' granules: k
// times the largest below the last.  For all threads.
template <class F, int NT, class S>
__device__ __noinline__ void top_by_rounds(S &sh, const Row<F> &row, const Share &share, int k) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t last = ~0ull;
    for (int r = 0; r < k; ++r) {
        uint64_t best = 0u;
        for (int g = share.g0 + tid; g < share.g1; g += NT) {
            float v[F::kElems];
            widen<F>(row.fetch(g), v);
            const uint32_t there = row.there(g);
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
        for (int w = 0; w < NT / 32; ++w)
            if (sh.best[w] > best) best = sh.best[w];
        if (tid == 0) sh.top[r] = best;
        last = best;
        __syncthreads();
    }
}

// Entries of a list of n, an even number, that are larger than e.
__device__ __forceinline__ int larger(const uint64_t *list, int n, uint64_t e) {
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(list + j);
        r += (v.x > e ? 1 : 0) + (v.y > e ? 1 : 0);
    }
    return r;
}

// Entries of each of n descending lists that are larger than e, in all.
__device__ __forceinline__ int larger(const uint64_t (&lists)[kMostCluster][kMostTop], int n, uint64_t e) {
    int at[kMostCluster];
#pragma unroll
    for (int o = 0; o < kMostCluster; ++o) at[o] = 0;
#pragma unroll 1
    for (int step = kMostTop / 2; step > 0; step >>= 1)
#pragma unroll
        for (int o = 0; o < kMostCluster; ++o)
            at[o] += lists[o][at[o] + step - 1] > e ? step : 0;
    int r = 0;
#pragma unroll
    for (int o = 0; o < kMostCluster; ++o)
        if (o < n) r += at[o] + (lists[o][at[o]] > e ? 1 : 0);
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Notes a thread's largest of each run of batches: 1 << shift of them, so that there are
// kRuns at most.
template <class F, int NT>
struct Runs {
    int shift, batch;
    float top;  // of the run under way

    __device__ __forceinline__ explicit Runs(int batches) : shift(0), batch(0), top(-INFINITY) {
        while ((batches + (1 << shift) - 1) >> shift > kRuns<F, NT>) ++shift;
    }
    template <class S>
    __device__ __forceinline__ void note(S &sh, float most) {
        top = max_nan(top, most);
        store_one<F>(&sh.slots[batch >> shift][threadIdx.x], top);
        ++batch;
        if ((batch & ((1 << shift) - 1)) == 0) top = -INFINITY;
    }
    // of a thread that noted all its batches
    __device__ __forceinline__ int count() const { return (batch + (1 << shift) - 1) >> shift; }
};

// Joins what the block's threads found; returns it in warp 0.  With k > 0 the block's largest
// are in sh.top behind the next barrier.
template <class F, int NT, class S>
__device__ __forceinline__ RowPart join_threads(S &sh, const Row<F> &row, const Share &share,
                                                Running<F> &run, const Runs<F, NT> &runs, int k, float c) {
    constexpr int WARPS = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the block's maximum, and the lowest thread that has it
    const uint32_t key = share.w0 + tid < share.w1 || share.end_of(tid) >= 0 ? ordered(run.top) : 0u;
    sh.keys[tid] = key;
    if (__syncthreads_or(run.shallow)) {
        const float2 zs = sums_again<F, NT>(row.x, row.V, run.top, share, c);
        run.z = Pair::of(zs.x, 0.0f);
        run.s = Pair::of(zs.y, 0.0f);
        run.shallow = true;
    }
    // one of 32 groups of threads a lane, in every warp alike
    uint32_t group_key = 0u;
    int group_owner = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const uint32_t v = sh.keys[w * 32 + lane];
        if (v > group_key) {
            group_key = v;
            group_owner = w * 32 + lane;
        }
    }
    const uint32_t top_key = __reduce_max_sync(0xffffffffu, group_key);
    const int owner = static_cast<int>(
        __reduce_min_sync(0xffffffffu, group_key == top_key && top_key != 0u ? static_cast<uint32_t>(group_owner) : NT));
    const float m = top_key == 0u ? -INFINITY : value_of(top_key);
    {
        // t by the block's maximum: as the reference stands to it, or the thread's own
        const float up = run.shallow ? (run.top - m) * c : -fmaf(m, c, -run.r);
        const float shift = fmaxf(up, -kDeep), f = exp2_fast(shift);
        float z = run.z.sum(), s = f * fmaf(shift, z, run.s.sum());
        z *= f;
        if (run.top == -INFINITY) z = s = 0.0f;
        // its sum is 1 and what may be little beside it
        if (tid == owner) {
            sh.owner_z = z;
            sh.owner_s = s;
            z = s = 0.0f;
        }
        z = warp_sum(z);
        s = warp_sum(s);
        if (lane == 0) {
            sh.z[warp] = z;
            sh.s[warp] = s;
        }
    }
    // The least of k groups' largest, those that rank first: k elements are no less.  Threads
    // whose largest is no less hold them all: about as many threads.  (1 where fewer groups
    // than k have an element; in the rank the lane stands in the last five bits, so that no
    // two are equal.)
    uint32_t least = 1u;
    if (k > 0) {
        const uint32_t mine = (group_key & ~31u) | (31u - lane);
        sh.groups[warp][lane] = mine;
        __syncwarp();
        int above = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint4 v = *reinterpret_cast<const uint4 *>(&sh.groups[warp][4 * j]);
            above += (v.x > mine ? 1 : 0) + (v.y > mine ? 1 : 0) + (v.z > mine ? 1 : 0) + (v.w > mine ? 1 : 0);
        }
        least = max(1u, __reduce_min_sync(0xffffffffu, above < k ? group_key : 0xFFFFFFFFu));
        // Their runs that hold them: one at least for each such thread (a NaN is looked at).
        // (Four at a time: one after another it took 7000 clocks while others read, of 32 runs.)
        if (key >= least) {
            const float low = value_of(least);
            uint32_t hit = 0u;
#pragma unroll 1
            for (int r0 = 0; r0 < runs.count(); r0 += 4)  // (there is place for a multiple of 4)
#pragma unroll
                for (int r = r0; r < r0 + 4; ++r) hit |= F::one(sh.slots[r][tid]) < low ? 0u : 1u << r;
            hit &= (1u << (runs.count() - 1) << 1) - 1u;
            const bool end = share.end_of(tid) >= 0 && !(sh.ends[tid] < low);
            int at = atomicAdd(&sh.items, __popc(hit) + (end ? 1 : 0));
#pragma unroll 1
            for (; hit; hit &= hit - 1, ++at)
                if (at < kItems) sh.item[at] = (__ffs(hit) - 1) << 10 | tid;
            if (end && at < kItems) sh.item[at] = kRuns<F, NT> << 10 | tid;
        }
    }
    __syncthreads();
    if (k > 0) {
        const int items = sh.items;
        if (items <= kItems) {
            constexpr int kLog2Batch = kRowBatch == 4 ? 2 : (kRowBatch == 2 ? 1 : 0);
            const int log2_per = kLog2Batch + runs.shift;  // granules of a run
            const int n = items << log2_per;
            const auto granule = [&](int i) {  // or -1
                const int what = sh.item[i >> log2_per], who = what & 1023, r = what >> 10;
                const int j = i & ((1 << log2_per) - 1);
                if (r == kRuns<F, NT>) return j == 0 ? share.end_of(who) : -1;
                const int g = share.w0 + who + ((r << log2_per) + j) * NT;
                return g < share.w1 ? g : -1;
            };
#pragma unroll 1
            for (int i = tid; i < n; i += NT) {
                const int g = granule(i);
                if (g >= 0) push<F>(sh, row, g, least, false);
            }
            __syncthreads();
        }
        if (items > kItems || sh.listed > kList) list_many<F, NT>(sh, row, share, key, least, k);
        const int n = sh.listed;
        if (n <= kList) {
            if (tid == 0) sh.list[n] = 0u;
            __syncthreads();
#pragma unroll 1
            for (int i = tid; i < n; i += NT) {
                const uint64_t me = sh.list[i];
                const int r = larger(sh.list, (n + 1) & ~1, me);
                if (r < k) sh.top[r] = me;
            }
        } else {
            top_by_rounds<F, NT>(sh, row, share, k);
        }
    }
    RowPart all = {top_key, 0.0f, 0.0f};
    if (warp != 0) return all;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        all.rest += sh.z[w];
        all.sum_t += sh.s[w];
    }
    if (owner >= NT) return all;
    const float oz = sh.owner_z;
    // (one token is 1 off by 2^-21 at most, two that are equal are 2 off by that: 1.5 tells them apart)
    if (all.rest + oz >= 1.5f) {
        all.rest += oz - 1.0f;
        all.sum_t += sh.owner_s;
        return all;
    }
    // one token holds more than two thirds of the sum: its thread's others once more, alone
    float r = 0.0f, q = 0.0f;
    const auto others = [&](int g) {
        float v[F::kElems];
        widen<F>(row.fetch(g), v);
#pragma unroll
        for (int e = 0; e < F::kElems; ++e)
            if (v[e] < m) {
                const float x = fmaxf((v[e] - m) * c, -kDeep), p = exp2_fast(x);
                r += p;
                q = fmaf(p, x, q);
            }
    };
    // (one body: the last turn of lane 0 is the row's end)
    const int end = lane == 0 ? share.end_of(owner) : -1;
    bool more = true;
#pragma unroll 1
    for (int g = share.w0 + owner + lane * NT; more; g += 32 * NT) {
        more = g < share.w1;
        if (!more) g = end;
        if (g >= 0) others(g);
    }
    all.rest += warp_sum(r);
    all.sum_t += warp_sum(q);
    return all;
}

// A row's results, by warp 0.
template <class S>
__device__ __forceinline__ void store_row(const LogprobsArgs &a, const S &sh, const RowPart &all, int64_t t,
                                          int64_t target, float given) {
    const int lane = threadIdx.x & 31;
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const float most = value_of(all.key), ln_z = log1pf(all.rest);
    const bool plain = fabsf(most) < INFINITY;
    const auto logp = [&](float x) {
        if (plain) return (x - most) * a.scale - ln_z;
        if (most == -INFINITY) return -INFINITY;
        return x < INFINITY && most == INFINITY ? -INFINITY : nan;
    };
    if (lane == 0) {
        const float none = most == -INFINITY ? 0.0f : nan;
        if (a.lse) a.lse[t] = plain ? fmaf(most, a.scale, ln_z) : most;
        if (a.entropy) a.entropy[t] = plain ? fmaf(-0.6931471805599453f, all.sum_t / (1.0f + all.rest), ln_z) : none;
        if (a.logprobs) {
            float v = 0.0f;
            if (target >= a.V) {
                atomicOr(&g_logprobs_status, RN_STATUS_BAD_INDEX);
                v = nan;
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

// The row's ends, by their threads.
template <class F, class S>
__device__ __forceinline__ void take_end(S &sh, const Row<F> &row, const Share &share, Running<F> &run,
                                         float c) {
    const int end = share.end_of(threadIdx.x);
    if (end < 0) return;
    const uint4 u[1] = {row.fetch(end)};
    const float most = largest<F>(u);
    run.take(u, most, c);
    sh.ends[threadIdx.x] = most;
}

// ---- the stream of batches ------------------------------------------------------------

// A block's share of its rows (t, t + step, ..) as one stream of batches.  Each thread
// copies its own granules to its own places in shared memory, kStages - 1 batches ahead of
// the one it takes, so that nothing waits for another thread, and the next row comes in
// while a row is joined.
template <class F, int NT, class S>
struct Stream {
    const LogprobsArgs &a;
    S &sh;
    const void *at;      // this thread's first granule of the batch to be copied next
    int left;            // granules of the share from the block's first of that batch on
    int rank;
    uint32_t head;       // stage of the batch to be copied next
    int64_t t, step;

    __device__ __forceinline__ Stream(const LogprobsArgs &a_, S &sh_, int rank_, int64_t t_, int64_t step_)
        : a(a_), sh(sh_), rank(rank_), head(0), t(t_), step(step_) {
        begin();
    }
    __device__ __forceinline__ void begin() {
        const Row<F> row(a.logits, a.stride, t, a.V);
        const Share share = Share::of(row, rank, a.blocks);
        at = row.x + row.index(share.w0 + threadIdx.x);
        left = share.w1 - share.w0;
    }
    // Copies a batch that is whole and not its share's last.
    __device__ __forceinline__ void copy_whole() {
        const uint8_t *from = static_cast<const uint8_t *>(at);
        uint4 *to = &sh.stage[head][0][threadIdx.x];
#pragma unroll
        for (int b = 0; b < kRowBatch; ++b) copy_async16(to + b * NT, from + b * NT * 16);
        at = from + kRowBatch * NT * 16;
        copy_commit();
        head = head + 1 == kStages<NT> ? 0 : head + 1;
    }
    // Copies a batch, if there is one; the group counts anyway.  (A share without a whole
    // granule is a batch of nothing.)
    __device__ __forceinline__ void copy() {
        if (t < a.T) {
            const uint8_t *from = static_cast<const uint8_t *>(at);
            uint4 *to = &sh.stage[head][0][threadIdx.x];
            if (left >= kRowBatch * NT) {
#pragma unroll
                for (int b = 0; b < kRowBatch; ++b) copy_async16(to + b * NT, from + b * NT * 16);
            } else {
#pragma unroll
                for (int b = 0; b < kRowBatch; ++b)
                    if (b * NT + static_cast<int>(threadIdx.x) < left) copy_async16(to + b * NT, from + b * NT * 16);
            }
            left -= kRowBatch * NT;
            at = from + kRowBatch * NT * 16;
            if (left <= 0) {
                t += step;
                if (t < a.T) begin();
            }
        }
        copy_commit();
        head = head + 1 == kStages<NT> ? 0 : head + 1;
    }
};

template <class F, int NT, bool CLUSTER>
__global__ void __launch_bounds__(NT, resident_blocks(NT)) logprobs_fwd_kernel(const __grid_constant__ LogprobsArgs a) {
    extern __shared__ __align__(16) uint8_t row_shared[];
    using S = RowShared<F, NT, CLUSTER>;
    S &sh = *reinterpret_cast<S *>(row_shared);
    pdl_trigger();
    if constexpr (CLUSTER) cluster_arrive();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x % a.blocks) : 0;
    const int64_t first = CLUSTER ? blockIdx.x / a.blocks : blockIdx.x;
    const int64_t step = CLUSTER ? gridDim.x / a.blocks : gridDim.x;
    Stream<F, NT, S> stream(a, sh, rank, first, step);
#pragma unroll 1
    for (int i = 0; i < kStages<NT> - 1; ++i) stream.copy();
    if (tid == 0) sh.listed = sh.items = 0;
    if (tid < kMostTop) sh.top[tid] = 0u;
    const float c = a.scale_log2;
    uint32_t tail = 0;  // stage of the batch to be taken next
    int turn = 0;       // of the two places for what the cluster knows

    for (int64_t t = first; t < a.T; t += step, turn ^= 1) {
        const Row<F> row(a.logits, a.stride, t, a.V);
        const Share share = Share::of(row, rank, a.blocks);
        // the given token's logit comes while the row is read
        int64_t target = -1;
        float given = 0.0f;
        if (rank == 0 && tid == 0 && a.targets) {
            target = a.targets[t];
            if (target >= 0 && target < a.V) given = F::one(row.x[target]);
        }
        Running<F> run;
        Runs<F, NT> runs((share.w1 - share.w0 + kRowBatch * NT - 1) / (kRowBatch * NT));
        take_end(sh, row, share, run, c);
        int g = share.w0;
        const auto taken = [&](const uint4 (&u)[kRowBatch]) {
            const float most = largest<F>(u);
            run.take(u, most, c);
            if (a.k > 0) runs.note(sh, most);
            g += kRowBatch * NT;
        };
        // while this batch and that to be copied are whole, and more of the share follows
        for (int n = (share.w1 - share.w0 - 1) / (kRowBatch * NT) - (kStages<NT> - 1); n > 0; --n) {
            copy_wait<kStages<NT> - 2>();
            uint4 u[kRowBatch];
            const uint4 *from = &sh.stage[tail][0][tid];
#pragma unroll
            for (int b = 0; b < kRowBatch; ++b) u[b] = ld_shared16(from + b * NT);
            tail = tail + 1 == kStages<NT> ? 0 : tail + 1;
            stream.copy_whole();
            stream.left -= kRowBatch * NT;
            taken(u);
        }
        do {
            copy_wait<kStages<NT> - 2>();
            uint4 u[kRowBatch];
            const uint4 *from = &sh.stage[tail][0][tid];
            if (g + kRowBatch * NT <= share.w1) {
#pragma unroll
                for (int b = 0; b < kRowBatch; ++b) u[b] = ld_shared16(from + b * NT);
            } else {
#pragma unroll
                for (int b = 0; b < kRowBatch; ++b) {
                    u[b] = make_uint4(F::kNone, F::kNone, F::kNone, F::kNone);
                    if (g + b * NT + tid < share.w1) u[b] = ld_shared16(from + b * NT);
                }
            }
            tail = tail + 1 == kStages<NT> ? 0 : tail + 1;
            stream.copy();  // (to the stage that the batch before came from)
            taken(u);
        } while (g < share.w1);
        RowPart all = join_threads<F, NT>(sh, row, share, run, runs, a.k, c);
        __syncthreads();
        if constexpr (CLUSTER) {
            // Everything goes to the first block, which joins it in the blocks' order.  The
            // barrier's phases: all have begun; then for each row: all have told, and the
            // first block has joined the row before, so the one behind may take its place.
            if (rank != 0 || t == first) cluster_wait();
            ClusterShared *to = cg::this_cluster().map_shared_rank(&sh.cluster, 0);
            if (tid == 0) to->parts[turn][rank] = all;
            if (tid < kMostTop && a.k > 0) to->tops[turn][rank][tid] = sh.top[tid];
            cluster_arrive();
            if (rank != 0) {
                if (tid < kMostTop) sh.top[tid] = 0u;
                if (tid == 0) sh.listed = sh.items = 0;
                continue;
            }
            cluster_wait();
            const int n = a.blocks;
            if (a.k > 0)
#pragma unroll 1
                for (int i = tid; i < n * kMostTop; i += NT) {
                    const uint64_t me = sh.cluster.tops[turn][i / kMostTop][i % kMostTop];
                    if (me == 0u) continue;
                    const int r = larger(sh.cluster.tops[turn], n, me);
                    if (r < a.k) sh.top[r] = me;
                }
            __syncthreads();
            if (warp == 0) {
                const RowPart p = lane < n ? sh.cluster.parts[turn][lane] : RowPart{0u, 0.0f, 0.0f};
                const uint32_t most = __reduce_max_sync(0xffffffffu, p.key);
                const int holder = __ffs(__ballot_sync(0xffffffffu, p.key == most)) - 1;
                float z = 0.0f, s = 0.0f;
                if (p.key != 0u) {
                    const float shift = fmaxf((value_of(p.key) - value_of(most)) * c, -kDeep), f = exp2_fast(shift);
                    s = f * fmaf(shift, 1.0f + p.rest, p.sum_t);
                    z = lane == holder ? p.rest : f * (1.0f + p.rest);
                }
                all = {most, warp_sum(z), warp_sum(s)};
            }
        }
        if (warp == 0) {
            store_row(a, sh, all, t, target, given);
            // for the next row; the others come to them behind its first barrier
            __syncwarp();
            sh.top[tid] = 0u;
            if (tid == 0) sh.listed = sh.items = 0;
        }
    }
    if (CLUSTER && rank != 0) cluster_wait();
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
    int share;       // granules of a block
};

constexpr int kGradThreads = 256;
constexpr int kGradBatch = 4;  // granules of a thread
// Beyond this the rounding of lse may put scale x - lse far above zero: 1e30 above in a row of
// nothing but bf16's or fp32's lowest value, and the power would be infinite.  There scale x is
// rounded before lse is taken off: no rounded s is above the rounded lse, so p is 1 at most.
constexpr float kFarLse = 0x1p20f;

// The granule of elements i .. of a row, wherever they lie: two aligned ones, shifted.
template <class F>
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, uint32_t bytes) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t s[6], q[5];
#pragma unroll
    for (int j = 0; j < 6; ++j) s[j] = bytes & 8u ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) q[j] = bytes & 4u ? s[j + 1] : s[j];
    const uint32_t bits = (bytes & 2u) * 8u;
    return make_uint4(__funnelshift_r(q[0], q[1], bits), __funnelshift_r(q[1], q[2], bits),
                      __funnelshift_r(q[2], q[3], bits), __funnelshift_r(q[3], q[4], bits));
}

// A block takes a share of a row, by the granules of dlogits; logits may lie otherwise
// within 16 bytes.  HBM bounds it: 4096 rows of 131072 in bf16, 2.15 GB, take 302 us (7.1 TB/s,
// 1.05 of the copy's rate) launch after launch, 319 a single call (0.99); 309 with loads and stores that keep their lines, 387 with two
// granules a thread, 351 with scalar fp32 and shares that leave each row's last block a rest.
// 2048 rows of 50021: 63 us (floor 60); 79 where dlogits lies otherwise than logits (235 with
// stores of one element).  40 registers a thread are six blocks an SM; with 46, five, the two
// take 307 and 65.
template <class F>
__global__ void __launch_bounds__(kGradThreads) logprobs_bwd_kernel(const __grid_constant__ LogprobsGradArgs a) {
    pdl_trigger();
    pdl_wait();
    const int64_t t = blockIdx.x / a.chunks;
    const int chunk = static_cast<int>(blockIdx.x - t * a.chunks);
    const Row<F> out(a.dlogits, a.dstride, t, a.V);
    const typename F::T *x = static_cast<const typename F::T *>(a.logits) + t * a.stride;
    typename F::T *y = const_cast<typename F::T *>(out.x);
    const int first = chunk * a.share + threadIdx.x;
    const int end = min(out.granules, (chunk + 1) * a.share);
    // granules g of which logits' 16 bytes (32 where they lie otherwise) are all the row's
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x + out.index(0))) & 15u;
    const int before = static_cast<int>(off / sizeof(typename F::T));
    const auto inside = [&](int g) {
        const int i = out.index(g) - before;
        return i >= 0 && i <= a.V - (off ? 2 : 1) * F::kElems;
    };
    uint4 u[kGradBatch];
#pragma unroll
    for (int b = 0; b < kGradBatch; ++b) {
        const int g = first + b * kGradThreads;
        u[b] = make_uint4(0u, 0u, 0u, 0u);
        if (g >= end) continue;
        const int i = out.index(g);
        if (!inside(g)) {
            u[b] = end_of_row<F>(x, i, static_cast<int>(a.V));
        } else if (off == 0u) {
            u[b] = ld_stream16(x + i);
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(x + (i - before));
            u[b] = shifted<F>(p[0], p[1], off);
        }
    }
    const float lse = a.lse[t];
    const float h = a.entropy ? a.entropy[t] : 0.0f;
    float dh = a.dentropy ? a.dentropy[t * a.dentropy_stride] : 0.0f;
    float dl = a.dlse ? a.dlse[t * a.dlse_stride] : 0.0f;
    int64_t wanted = -1;
    float dp = 0.0f, lt = 0.0f;
    if (a.dlogprobs) {
        wanted = a.targets[t];
        if (wanted >= 0) {
            dp = a.dlogprobs[t * a.dlogprobs_stride];
            lt = a.logprobs[t];
        }
    }
    const float nan = __uint_as_float(0x7FFFFFFFu);
    if (lse == -INFINITY) dp = dh = dl = 0.0f;  // all tokens are banned, or too far down for fp32
    if (!(lse < INFINITY)) dp = nan;            // NaN or +infinity
    // (-1: none of the row's)
    const int target = wanted < a.V ? static_cast<int>(wanted < 0 ? -1 : wanted) : -1;
    if (wanted >= a.V) {
        dp = nan;
        if (chunk == 0 && threadIdx.x == 0) atomicOr(&g_logprobs_status, RN_STATUS_BAD_INDEX);
    }
    // dx = p (c0 - c1 (s - lse)); s - lse stops at -150, where p is zero and a product with
    // the -infinity of a banned token would be NaN
    const float c0 = a.scale * (dl - dp - dh * h), c1 = a.scale * dh;
    // of the given token, by its own log probability: 1 - p where p is nearly 1
    const auto given = [&] {
        const float l = fmaxf(lt, -150.0f);
        return a.scale * (expf(l) * (dl - dh * (l + h)) - expm1f(l) * dp);
    };
    const Pair scale = Pair::both(a.scale), log2e = Pair::both(1.4426950408889634f);
    const Pair k0 = Pair::both(c0), k1 = Pair::both(-c1);
    const auto grad = [&](float &p, float &q, Pair ref, auto far) {
        float2 l = Pair::of(p, q).fma(scale, ref).v;
        if constexpr (far.value)  // (scalar operations: a packed product and sum may become one)
            l = make_float2(__fadd_rn(__fmul_rn(p, a.scale), ref.v.x), __fadd_rn(__fmul_rn(q, a.scale), ref.v.y));
        const Pair m = Pair::of(fmaxf(l.x, -150.0f), fmaxf(l.y, -150.0f));
        const float2 e = (m * log2e).v;
        const float2 r = (Pair::of(exp2_fast(e.x), exp2_fast(e.y)) * m.fma(k1, k0)).v;
        p = r.x;
        q = r.y;
    };
    // (both ways whole: a choice within the loop takes registers of the usual one)
    const auto store = [&](Pair ref, auto far) {
#pragma unroll
        for (int b = 0; b < kGradBatch; ++b) {
            const int g = first + b * kGradThreads;
            if (g >= end) return;
            const int i = out.index(g);
            float v[F::kElems];
            widen<F>(u[b], v);
#pragma unroll
            for (int e = 0; e < F::kElems; e += 2) grad(v[e], v[e + 1], ref, far);
            if (target >= 0 && static_cast<uint32_t>(target - i) < F::kElems) {
                const float gt = given();
#pragma unroll
                for (int e = 0; e < F::kElems; ++e)
                    if (target == i + e) v[e] = gt;
            }
            if (out.whole(g)) {
                __stcs(reinterpret_cast<uint4 *>(y + i), narrow<F>(v));
            } else {
                const uint32_t there = out.there(g);
#pragma unroll
                for (int e = 0; e < F::kElems; ++e)
                    if (there >> e & 1u) store_one<F>(y + i + e, v[e]);
            }
        }
    };
    if (!(fabsf(lse) > kFarLse))
        store(Pair::both(-lse), std::false_type());
    else  // (-infinity: p is 0)
        store(Pair::both(lse == -INFINITY ? lse : -lse), std::true_type());
}

// ---- host ---------------------------------------------------------------------------------------

static int elem_bytes(int dtype) { return dtype == RN_DTYPE_F32 ? 4 : 2; }

// Threads of a block, and blocks that share a row.
struct RowShape {
    int threads, blocks;
};
// The layout that an estimate prefers.  An SM takes its blocks' shares of rows in rounds of
// as many as it holds.  A round takes what HBM needs for the SM's shares in it (44.6 KB a us),
// what a block needs to take in its own (3.2 KB a us for each warp), and some us in which rows
// are joined; clusters do not fill all SMs alike.  So many rows are best in rounds that are
// nearly full, few rows on many blocks each.  Over the 159 pairs of T and V in three formats that
// it was fitted to it chose layouts that took 2.8% longer than the best of them on average, 23% at
// most; over 217 others 4.9%, and 37% (100 fp16 rows of 50021 without alternatives: 8.9 us in
// blocks of 320, 6.5 in clusters of 8 x 128).  It does not know how many alternatives a join
// looks for: without any, clusters are better further up than it says.
// (8 alternatives, bf16, 131072 columns, us as 512 threads x 1 block / 256 x 1 / 128 x 1 / 96 x 1 /
// 64 x 1 / 128 x 4 / 128 x 8 / 256 x 8; * what it chooses.  64 rows 12.1 / 14.8 / 15.2 / 29.7 / 38.5 / 11.1 /
// 11.6 / 10.9*; 76 10.8 / 15.0 / 15.4 / 29.8 / 38.6 / 11.7 / 11.8* / 14.9; 152 12.1* / 15.7 / 16.1 / 29.0 / 37.0 / 14.7 /
// 20.7 / 28.7; 500 30.8 / 26.6* / 32.8 / 35.9 / 44.7; 1000 59.0 / 52.6 / 46.7* / 57.9 / 63.4; 1500 75.5 / 78.6 / 80.1 /
// 65.9* / 72.7; 2048 104 / 104 / 91.2 / 115 / 86.9*; 3000 146 / 132 / 133 / 129* / 155.)
static RowShape row_shape(int64_t T, int64_t V, int dtype, int sm_count) {
    const double kb = static_cast<double>(V) * elem_bytes(dtype) / 1024;
    RowShape best = {256, 1};
    double least = 0;
    for (int threads : {512, 320, 256, 192, 128, 96, 64}) {
        double join = 3.5 + threads / 150.0;
        for (int blocks : {1, 4, kMostCluster}) {
            // clusters of blocks of 128 or 256; two granules a thread at least
            if (blocks > 1 && ((threads != 128 && threads != 256) || kb * 64 < 2.0 * threads * blocks)) break;
            join += blocks == 1 ? 0.0 : blocks == 4 ? 2.75 : 0.25;
            // (their shared memory counts, too, and not every place suits a cluster)
            const double resident = blocks == 1 ? resident_blocks(threads) : threads == 128 ? 5.7 : 3.8;
            const double each = static_cast<double>(T) * blocks / sm_count;
            const double rounds = ceil(each / resident), at_once = ceil(each / rounds);
            const double us =
                rounds * (kb / blocks * (at_once / 44.6 + 10.0 / threads) * (blocks > 1 ? 1.5 : 1.0) + join);
            if (least == 0 || us < least) {
                least = us;
                best = {threads, blocks};
            }
        }
    }
    return best;
}

template <class F, int NT, bool CLUSTER>
static int launch_fwd(const LogprobsArgs &a, const DeviceInfo &dev, cudaStream_t st) {
    static std::atomic<int> resident[kMaxDevices];  // blocks that an SM holds
    const auto kernel = logprobs_fwd_kernel<F, NT, CLUSTER>;
    constexpr int smem = sizeof(RowShared<F, NT, CLUSTER>);
    const int idx = current_device_index();
    if (idx < 0 || idx >= kMaxDevices) return RN_ERR_DEVICE;
    int fit = resident[idx].load(std::memory_order_acquire);
    if (fit == 0) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, NT, smem) != cudaSuccess || fit < 1) {
            cudaGetLastError();
            return RN_ERR_DEVICE;
        }
        resident[idx].store(fit, std::memory_order_release);
    }
    // as many rows at once as the GPU holds
    int64_t rows = static_cast<int64_t>(dev.sm_count) * fit / a.blocks;
    if (rows > a.T) rows = a.T;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * a.blocks));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.blocks);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return RN_ERR_LAUNCH;
    }
    return cudaGetLastError() == cudaSuccess ? RN_OK : RN_ERR_LAUNCH;
}

template <class F>
static int run_fwd(LogprobsArgs &a, int dtype, const DeviceInfo &dev, cudaStream_t st) {
    const RowShape s = row_shape(a.T, a.V, dtype, dev.sm_count);
    a.blocks = s.blocks;
    switch (s.threads) {
        case 512: return launch_fwd<F, 512, false>(a, dev, st);
        case 320: return launch_fwd<F, 320, false>(a, dev, st);
        case 192: return launch_fwd<F, 192, false>(a, dev, st);
        case 96: return launch_fwd<F, 96, false>(a, dev, st);
        case 64: return launch_fwd<F, 64, false>(a, dev, st);
        case 128: return a.blocks > 1 ? launch_fwd<F, 128, true>(a, dev, st) : launch_fwd<F, 128, false>(a, dev, st);
        default: return a.blocks > 1 ? launch_fwd<F, 256, true>(a, dev, st) : launch_fwd<F, 256, false>(a, dev, st);
    }
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
    a.logprobs = logprobs;
    a.lse = lse;
    a.entropy = entropy;
    a.top_logprobs = top_logprobs;
    a.top_ids = top_ids;
    const auto st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == RN_DTYPE_F32) return rn::run_fwd<rn::Row32>(a, dtype, *dev, st);
    if (dtype == RN_DTYPE_F16) return rn::run_fwd<rn::Row16Half>(a, dtype, *dev, st);
    return rn::run_fwd<rn::Row16Bf>(a, dtype, *dev, st);
}

int token_logprobs_select_layout(int dtype, int64_t T, int64_t V, int *threads, int *blocks) {
    const int rc = rn::check_rows(dtype, V, T, V, 1.0f);
    if (rc != RN_OK) return rc;
    if (T < 1) return RN_ERR_SHAPE;
    if (!threads || !blocks) return RN_ERR_NULL;
    const rn::DeviceInfo *dev = rn::current_device_info();
    if (!dev) return RN_ERR_DEVICE;
    const rn::RowShape s = rn::row_shape(T, V, dtype, dev->sm_count);
    *threads = s.threads;
    *blocks = s.blocks;
    return RN_OK;
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
    if (T > 1 && dlogits == logits && dlogits_stride != stride) return RN_ERR_ARG;  // in place is row by row
    const int64_t elems = 16 / bytes, per = static_cast<int64_t>(rn::kGradThreads) * rn::kGradBatch;
    rn::LogprobsGradArgs a = {};
    // (a row that begins inside a granule may touch one more)
    const bool inside = rn::misaligned(dlogits, 16) || (T > 1 && dlogits_stride * bytes % 16 != 0);
    const int64_t granules = (V + elems - 1) / elems + (inside ? 1 : 0);
    a.chunks = (granules + per - 1) / per;
    if (a.chunks > INT32_MAX / T) return RN_ERR_SHAPE;
    // equal shares, in whole warps' rounds
    a.share = static_cast<int>(((granules + a.chunks - 1) / a.chunks + 31) / 32 * 32);
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
