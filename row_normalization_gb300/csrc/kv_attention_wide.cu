// kv_attention_wide.cu -- attention of many queries a sequence over the quantised
// key/value cache (sm_103a): chunks of a prompt against what the cache holds.
//
// The same formula as kv_attention.cu with 128 columns (queries times heads of the
// group) at a time, which makes it a matter of arithmetic: 4 D flops for each
// column and token against one restored key and value.  The products run as
// tcgen05.mma with the columns as the 128 rows of the accumulator:
//   S = Q K'^T + Q K''^T   Q, K' and K'' in shared memory, S in tensor memory,
//   O += P V'              P in tensor memory (over its S), V' in shared memory.
// P and V' are fp16, the tensor cores' rate being half in tf32 and tensor memory full.
// V' is the cached value s * c rounded once to fp16, K' the same of the key and K''
// the exact rest, so the logits (and lse) have no rounding but that of fp32 sums.
// Queries as in kv_attention.cu.  A token with a scale so large that s * c would leave
// fp16 is restored at 2^-3 of its size (2^-7 in 8 bits), and its logit, or its weight,
// makes up for it; what it has beside that in scales 2^-11 (2^-7) and below loses bits.
//
// Roles: four warps for each query tile of 128 columns, one accumulator row a thread
// (softmax, output); four that restore keys, four for values; one thread issues the
// products.  Two query tiles share every restored tile and take turns: the products
// of one run beside the softmax of the other.
//
// What bounds it: 64 queries over 131072 tokens of 8 heads of 128 in 4 bits (two query
// tiles) take 247 us, 556 TFLOP/s: 9000 clocks a tile of 256 columns by 128 tokens,
// of which the products need 3000 and the exponentials (16 a clock and SM) 2000.  No
// unit is full (tensor cores about a third, issue slots a third): with an earlier form
// without K'' that took 8700 clocks, leaving out the restoring gave 7000, three
// quarters of the softmax 8300, most of the products 7100, all of these 2900.  What
// is left is each role's latency, the handing over between them, and registers: with two
// query tiles 17 warps are allotted as 20, 96 registers a thread, and up to 550 bytes a
// thread are spilled and reloaded (with one tile 13 warps have 128, and a tenth of that).
// How much code lies between the roles' loops shows as well: forms that differ in nothing
// that runs differ by 10%.
//
// Shared memory operands are K-major with the 128-byte exchange of 16-byte chunks
// (chunk ^ row % 8 in rows of 128 bytes): 64 elements a row, blocks of 64 elements
// one after the other.  In 4 bits the eight dimensions of a chunk lie in the order
// 0 4 1 5 2 6 3 7, the order in which they leave a word, in Q as in K' and K''.
#include <float.h>

#include "kv_attention.cuh"

namespace rn {

// Weights (times 2^kDown of a large token) stay below 2^kWideRoom.  They are fp16, and a new
// reference leaves them kWideSlack powers of two to grow before a rescale: the largest is
// 2^10 at least, so 2^-24 of it is a normal number.
constexpr float kWideRoom = 15.0f;
constexpr float kWideSlack = 4.0f;
constexpr long long kWideLimit = 4000000000ll;  // clocks a wait may take, about two seconds

// QT query tiles of 128 columns at a time: two share the restored tiles and take
// turns at the tensor cores, one softmax beside the other's products; one where there
// are no more columns, or no tensor memory for two (D 256).
template <int D, int BITS, int QT>
struct WideShape {
    using F = KvFormat<D, BITS>;
    // Tokens of a tile.  (D 128 with two query tiles: tiles of 64 would leave tensor
    // memory for two S each, but what a tile costs beside its tokens outweighs that: in an
    // earlier form, without K'', 64 queries over 131072 tokens of 8 heads 289 against 257
    // us.)
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int kBufs = QT * (2 * BN + D) <= 512 ? 2 : 1;  // S of a query tile
    static constexpr int kStages = 2;                                              // of values
    static constexpr int kKeyStages = (D == 128 && QT == 2) || D == 256 ? 1 : 2;  // what fits
    static constexpr int NQ = 128 * QT;
    using L = LineShape<NQ, BN, 4, 1>;
    static constexpr int kWarps = 4 * QT + 9;        // softmax, keys, values, products
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kQuery = 128 * D * 2;       // a query tile
    static constexpr int kStage = BN * D * 2;        // a tile's values
    static constexpr int kKeyStage = 2 * kStage;     // its keys, and what rounding them left
    static constexpr int kUsed = 1024 + QT * kQuery + kKeyStages * kKeyStage + kStages * kStage;
    // more than half of an SM's shared memory: the tensor memory of an SM has one owner
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static constexpr int kSlot = NQ * (D + 2);
    // tensor memory columns: the S buffers, then O
    static constexpr uint32_t kO = QT * kBufs * BN;
    static_assert(kO + QT * D <= 512 && kUsed <= 226 * 1024, "tensor and shared memory");
    static_assert(QT * kBufs <= 2 && kKeyStages <= 2 && kStages <= 2, "WideShared has barriers for two of each");
    // S buffer and barrier phase of a query tile's c-th tile of tokens
    __device__ static __forceinline__ uint32_t buf(uint32_t qt, uint32_t c) { return qt * kBufs + c % kBufs; }
    __device__ static __forceinline__ uint32_t phase(uint32_t c) { return c / kBufs & 1; }
    // stage and barrier phase of the CTA's n-th tile
    __device__ static __forceinline__ uint32_t stage(uint32_t n) { return n % kStages; }
    __device__ static __forceinline__ uint32_t round(uint32_t n) { return n / kStages & 1; }
    __device__ static __forceinline__ uint32_t key_stage(uint32_t n) { return n % kKeyStages; }
    __device__ static __forceinline__ uint32_t key_round(uint32_t n) { return n / kKeyStages & 1; }
};

// ---- tensor memory and tcgen05 ------------------------------------------------------

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// A shared memory operand: K-major, 128-byte exchange, 8 rows every 1024 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// fp16 operands, fp32 accumulator, 128 rows by n columns.
constexpr uint32_t wide_idesc(int n) {
    return (1u << 4) | (static_cast<uint32_t>(n / 8) << 17) | (static_cast<uint32_t>(128 / 16) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// 32 columns of the warp's 32 rows, one row a thread; the registers hold them after
// the next tmem_wait_load on them.
__device__ __forceinline__ void tmem_load32(uint32_t (&u)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr)
        : "memory");
}
// Waits for every load of the thread; u takes part so that no use of it comes before.
__device__ __forceinline__ void tmem_wait_load(uint32_t (&u)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]),
                   "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]),
                   "+r"(u[15]), "+r"(u[16]), "+r"(u[17]), "+r"(u[18]), "+r"(u[19]), "+r"(u[20]), "+r"(u[21]),
                   "+r"(u[22]), "+r"(u[23]), "+r"(u[24]), "+r"(u[25]), "+r"(u[26]), "+r"(u[27]), "+r"(u[28]),
                   "+r"(u[29]), "+r"(u[30]), "+r"(u[31])
                 :
                 : "memory");
}
// 16 columns, complete on return.
__device__ __forceinline__ void tmem_load16(uint32_t (&u)[16], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- small helpers --------------------------------------------------------------------

// Generic writes to shared memory become visible to the tensor core's reads.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// s0 += x0, s1 += x1 in one instruction.
__device__ __forceinline__ void add_pairs(float &s0, float &s1, float x0, float x1) {
    asm("{\n\t.reg .b64 s, x;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tadd.rn.f32x2 s, s, x;\n\t"
        "mov.b64 {%0, %1}, s;\n\t}"
        : "+f"(s0), "+f"(s1) : "f"(x0), "f"(x1));
}

// The bits below bit n (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1u); }

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }

// A word of eight 4-bit codes as four pairs (element n, n + 4), n = 0..3, of c - 8.
__device__ __forceinline__ void codes_of(uint32_t w, __half2 (&h)[4]) {
    const __half2 z = __float2half2_rn(1032.0f), r = __float2half2_rn(0.0625f), z2 = __float2half2_rn(-72.0f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t u = w >> (8 * i);
        h[2 * i] = __hsub2(as_h2((u & 0x000F000Fu) | 0x64006400u), z);            // 1024 + c
        h[2 * i + 1] = __hfma2(as_h2((u & 0x00F000F0u) | 0x64006400u), r, z2);    // 1024 + 16 c
    }
}
// Two words of eight 8-bit codes as four pairs of neighbours, of c - 128.
__device__ __forceinline__ void codes_of(uint32_t w0, uint32_t w1, __half2 (&h)[4]) {
    const __half2 z = __float2half2_rn(1152.0f);
    h[0] = __hsub2(as_h2(__byte_perm(w0, 0x64646464u, 0x4140)), z);
    h[1] = __hsub2(as_h2(__byte_perm(w0, 0x64646464u, 0x4342)), z);
    h[2] = __hsub2(as_h2(__byte_perm(w1, 0x64646464u, 0x4140)), z);
    h[3] = __hsub2(as_h2(__byte_perm(w1, 0x64646464u, 0x4342)), z);
}

template <int WORDS>
__device__ __forceinline__ void load_global(uint32_t (&w)[WORDS], const void *src) {
    const uint32_t *p = static_cast<const uint32_t *>(src);
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int k = 0; k < WORDS; k += 4) {
            const uint4 v = ld_ro16(p + k);
            w[k] = v.x;
            w[k + 1] = v.y;
            w[k + 2] = v.z;
            w[k + 3] = v.w;
        }
    } else if constexpr (WORDS == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x;
        w[1] = v.y;
    } else {
        static_assert(WORDS == 1, "one, two or a multiple of four words");
        w[0] = __ldg(p);
    }
}

// Scales above kBig (the largest s with s * Q inside fp16: 9352, 515.5), and NaN, take the
// slow way: the token counts at 2^-kDown.
template <int BITS>
struct Big {
    static constexpr uint32_t kBig = BITS == 4 ? 0x7091u : 0x6007u;
    static constexpr int kDown = BITS == 4 ? 3 : 7;
    static constexpr float kUp = static_cast<float>(1 << kDown);
    // Scales of a token, two a word: whether one is that large.  (Shifted by an exponent, so
    // that infinity and NaN are negative integers.)
    template <int N>
    __device__ static __forceinline__ bool some(const uint32_t (&s)[N]) {
        constexpr uint32_t kMost = (kBig + 0x0400u) * 0x00010001u;
        uint32_t m = kMost;
#pragma unroll
        for (int k = 0; k < N; ++k) m = __vmaxs2(m, (s[k] & 0x7FFF7FFFu) + 0x04000400u);
        return m != kMost;
    }
    template <int N>
    __device__ static __forceinline__ void down(uint32_t (&s)[N]) {
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] = h2_bits(__hmul2(as_h2(s[k]), __float2half2_rn(1.0f / kUp)));
    }
};

// Tokens t .. t + 31 that a row does not see, a bit each: behind its position pos, or
// before its window's first token lo and no sink.
__device__ __forceinline__ uint32_t hidden_tokens(int pos, int lo, int sinks, int t) {
    return ~below(pos + 1 - t) | (below(lo - t) & ~below(sinks - t));
}

// Large tokens are rare.  What the softmax does about them is two calls, by tensor memory:
// inlined into the loop over 32 tokens it cost every tile its place in the instruction
// caches (3 chunks of 500 to 1300 queries 426 us, as calls 359).
//
// In front of a tile's softmax: the products with large keys come up to their size.  Returns
// the row's largest logit with a large value, whose weight counts 2^DOWN.
template <int BN, int DOWN>
__device__ __noinline__ float large_logits(uint32_t sbase, const uint32_t *key_big, const uint32_t *val_big,
                                           float factor, int pos, int lo, int sinks, int t0) {
    float most = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < BN; i += 16) {
        const uint32_t up = key_big[i / 32] >> (i & 31);
        const uint32_t bound = (val_big[i / 32] & ~hidden_tokens(pos, lo, sinks, t0 + (i & ~31))) >> (i & 31);
        uint32_t x[16];
        tmem_load16(x, sbase + i);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float y = __uint_as_float(x[j]) * (up >> j & 1u ? static_cast<float>(1 << DOWN) : 1.0f);
            x[j] = __float_as_uint(y);
            if (bound >> j & 1u) most = fmaxf(most, fmaf(y, factor, DOWN));
        }
        tmem_store16(sbase + i, x);
    }
    tmem_wait_store();
    return most;
}
// Behind it: the weights of large values come up.
template <int BN, int DOWN>
__device__ __noinline__ void large_weights(uint32_t sbase, const uint32_t *val_big) {
    tmem_wait_store();
#pragma unroll 1
    for (int i = 0; i < BN / 32; ++i) {
        const uint32_t up = val_big[i];
        uint32_t x[16];
        tmem_load16(x, sbase + 16 * i);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t two = up >> (2 * j);
            x[j] = h2_bits(__hmul2(as_h2(x[j]), as_h2(0x3C003C00u + ((two & 1u) | (two & 2u) << 15) * (DOWN << 10))));
        }
        tmem_store16(sbase + 16 * i, x);
    }
}

// Brings stored weights, 32 of each of the tile's first `chunks` quarters, down by a power of
// two: in two steps, as it may be too small for fp16 where what it leaves of a weight is not.
__device__ __forceinline__ void scale_weights(uint32_t sbase, int chunks, float scale) {
    const uint32_t half = (127u - (__float_as_uint(scale) >> 23)) >> 1;
    const __half2 first = __float2half2_rn(__uint_as_float((127u - half) << 23));
    const __half2 second = __float2half2_rn(scale * __uint_as_float((127u + half) << 23));
    tmem_wait_store();
#pragma unroll 1
    for (int i = 0; i < 16 * chunks; i += 16) {
        uint32_t x[16];
        tmem_load16(x, sbase + i);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = h2_bits(__hmul2(__hmul2(as_h2(x[j]), first), second));
        tmem_store16(sbase + i, x);
    }
    tmem_wait_store();
}

struct WideShared {
    uint64_t q_full[2];                            // by query tile
    uint64_t k_full[2], v_full[2], k_free[2], v_free[2];  // by stage
    uint64_t s_full[2], p_full[2], pv_done[2];            // by S buffer
    uint64_t drained;
    uint32_t tmem;
    int abort;
    // What restoring a tile met, a byte for each of the four warps: 1 where a token counts
    // at 2^-kDown, 2 where a value is NaN; and those tokens, a bit each, 32 a word.  Keys:
    // their producers wait for the products of two tiles before, which wait for the softmax
    // of two tiles before that, so eight tiles' are kept.  Values: by stage.
    uint32_t key_flags[8], val_flags[2];
    uint32_t key_big[8][4], val_big[2][4];
    float large[256];  // by row: its largest logit with a large value of the tile, and kDown
    int64_t scratch[17 + 2];
};

// A wait with a limit; gives up for the whole CTA when it runs out.  (The limit is
// counted in SM clocks: reading the global timer in every wait costs more than the
// wait.)
__device__ __forceinline__ bool wide_wait(WideShared &sh, uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0) {
            if (*const_cast<volatile int *>(&sh.abort)) return false;
            if (clock64() - t0 > kWideLimit) break;
        }
    }
    if (atomicExch(&sh.abort, 1) == 0) atomicOr(&g_kv_attention_status, RN_STATUS_WAIT_TIMEOUT);
    return false;
}
// The same by a whole warp, which is together again afterwards.
__device__ __forceinline__ bool wide_wait_warp(WideShared &sh, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wide_wait(sh, bar, parity));
}

// What a thread needs to find a token's rows.
struct TokenRows {
    KvCache cache;
    const int32_t *table;  // of the sequence
    int kvh, hi, win_lo, sinks;

    template <class L>
    __device__ __forceinline__ TokenRows(const KvAttnArgs &a, const Item<L> &it, int head)
        : cache(a.cache), table(a.page_table + it.seq * a.max_pages), kvh(head), hi(it.hi), win_lo(it.win_lo),
          sinks(a.sinks) {}
    __device__ __forceinline__ bool seen(int t) const {
        return t < hi && (win_lo == 0 || t < sinks || t >= win_lo);
    }
    // Every (some) token of t .. t + 7 is seen.
    __device__ __forceinline__ bool all_seen(int t) const {
        return t + 7 < hi && (win_lo == 0 || t >= win_lo || t + 7 < sinks);
    }
    __device__ __forceinline__ bool some_seen(int t) const {
        return t < hi && (win_lo == 0 || t < sinks || t + 7 >= win_lo);
    }
    // The row of token t's key (which 0) or value, or -1 where its page does not exist.
    __device__ __forceinline__ int64_t row(int t, int which) const {
        const int page = table[t >> cache.log2_page];
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(cache.num_pages)) {
            atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
            return -1;
        }
        return cache.row(page, which, kvh, t & ((1 << cache.log2_page) - 1));
    }
};

// ---- restoring keys ---------------------------------------------------------------------
// Four warps, BN / 4 tokens each, eight at a time: lane = token % 8 + 8 j with j the
// quarter of the stored row.  A group's eight elements are one chunk of the operand.
// A key s * c has up to 18 significant bits: its fp16 and the exact rest, which the
// fused multiply-add gives, are two operands behind one another.
template <int D, int BITS, int BN>
struct KeyTile {
    using F = KvFormat<D, BITS>;
    static constexpr int ITER = BN / 32, KW = F::kGroups * BITS / 4, SW = F::kGroups / 2;
    uint32_t w[ITER][KW], s[ITER][SW];

    __device__ __forceinline__ void load(const TokenRows &rows, int t0, int warp, int lane) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int t = t0 + warp * (BN / 4) + 8 * i + (lane & 7);
            const int64_t r = rows.seen(t) ? rows.row(t, 0) : -1;
            if (r >= 0) {
                load_global<KW>(w[i], rows.cache.codes + r * F::kRow + (lane >> 3) * KW * 4);
                load_global<SW>(s[i], rows.cache.scales + r * F::kGroups);
            } else {
#pragma unroll
                for (int k = 0; k < KW; ++k) w[i][k] = 0u;
#pragma unroll
                for (int k = 0; k < SW; ++k) s[i][k] = 0u;
            }
        }
    }
    __device__ __forceinline__ bool special() const {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < ITER; ++i)
#pragma unroll
            for (int k = 0; k < SW; ++k) m = __vmaxu2(m, s[i][k]);
        return max(m & 0xFFFFu, m >> 16) > Big<BITS>::kBig;
    }
    __device__ __forceinline__ void store(uint8_t *stage, int warp, int lane) const {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int row = warp * (BN / 4) + 8 * i + (lane & 7);
#pragma unroll
            for (int g = 0; g < F::kGroups; ++g) {
                const __half2 pair = as_h2(s[i][g / 2]);
                const __half2 sc = g & 1 ? __high2half2(pair) : __low2half2(pair);
                __half2 h[4];
                if constexpr (BITS == 4)
                    codes_of(w[i][g], h);
                else
                    codes_of(w[i][2 * g], w[i][2 * g + 1], h);
                const int chunk = 4 * g + (lane >> 3);
                uint8_t *to = stage + (chunk >> 3) * (BN * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
                __half2 k[4], rest[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    k[e] = __hmul2(h[e], sc);
                    rest[e] = __hfma2(h[e], sc, __hneg2(k[e]));
                }
                *reinterpret_cast<uint4 *>(to) =
                    make_uint4(h2_bits(k[0]), h2_bits(k[1]), h2_bits(k[2]), h2_bits(k[3]));
                *reinterpret_cast<uint4 *>(to + BN * D * 2) =
                    make_uint4(h2_bits(rest[0]), h2_bits(rest[1]), h2_bits(rest[2]), h2_bits(rest[3]));
            }
        }
    }
    // Takes the large tokens down; returns a bit each of the warp's.  (A call, on a copy.)
    struct Scales {
        uint32_t s[ITER][SW];
    };
    __device__ __noinline__ static uint32_t tame(Scales &x, int lane) {
        uint32_t big = 0u;
#pragma unroll 1
        for (int i = 0; i < ITER; ++i)
            if (Big<BITS>::some(x.s[i])) {
                Big<BITS>::down(x.s[i]);
                big |= 1u << (8 * i + (lane & 7));
            }
        return __reduce_or_sync(0xffffffffu, big);
    }
    __device__ __forceinline__ uint32_t tame(int lane) {
        Scales x;
        memcpy(x.s, s, sizeof s);
        const uint32_t big = tame(x, lane);
        memcpy(s, x.s, sizeof s);
        return big;
    }
};

// ---- restoring values, transposed --------------------------------------------------------
// A thread takes eight tokens of the stored rows' r-th run (or half of it, 64 tokens) and
// writes, for each of its dimensions, the eight tokens as one chunk of that
// dimension's row.  r and the tokens are mixed over the lanes so that eight
// neighbours write eight different banks' chunks.
template <int D, int BITS, int BN>
struct ValueTile {
    using F = KvFormat<D, BITS>;
    static constexpr int SPLIT = BN == 64 ? 2 : 1;
    static constexpr int VW = D * BITS / 256 / SPLIT, SW = BITS == 4 ? VW : (VW + 1) / 2;
    uint32_t w[8][VW], s[8][SW];
    uint32_t other;  // the largest scales of the row's other part

    struct Place {
        int r, chunk, part;
    };
    __device__ static __forceinline__ Place place(int warp, int lane) {
        Place p;
        p.r = (lane & 3) | (lane >> 1 & 4);
        const int tg = (lane >> 2 & 1) | (lane >> 3 & 2);
        p.chunk = SPLIT == 2 ? (warp & 1) * 4 + tg : warp * 4 + tg;
        p.part = SPLIT == 2 ? warp >> 1 : 0;
        return p;
    }
    __device__ __forceinline__ void load(const TokenRows &rows, int t0, const Place &p) {
        const int t = t0 + 8 * p.chunk;
        const int64_t r = rows.some_seen(t) ? rows.row(t, 1) : -1;
        const bool all = rows.all_seen(t);
        other = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r >= 0 && (all || rows.seen(t + i))) {
                load_global<VW>(w[i], rows.cache.codes + (r + i) * F::kRow + (p.r * SPLIT + p.part) * VW * 4);
                uint32_t row[SPLIT * SW];
                load_global<SPLIT * SW>(row, rows.cache.scales + (r + i) * F::kGroups);
#pragma unroll
                for (int k = 0; k < SW; ++k) {
                    s[i][k] = p.part ? row[(SPLIT - 1) * SW + k] : row[k];
                    if constexpr (SPLIT == 2) other = __vmaxu2(other, p.part ? row[k] : row[SW + k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < VW; ++k) w[i][k] = 0u;
#pragma unroll
                for (int k = 0; k < SW; ++k) s[i][k] = 0u;
            }
        }
    }
    __device__ __forceinline__ bool special() const {
        uint32_t m = other;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < SW; ++k) m = __vmaxu2(m, s[i][k]);
        return max(m & 0xFFFFu, m >> 16) > Big<BITS>::kBig;
    }
    __device__ __forceinline__ void store(uint8_t *stage, const Place &p) const {
        uint8_t *base = stage + (p.chunk >> 3) * (D * 128);
        const auto put = [&](int d, const uint32_t (&v)[4]) {
            *reinterpret_cast<uint4 *>(base + d * 128 + (((p.chunk & 7) ^ (d & 7)) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
        };
        // scales of the tokens 2i, 2i + 1 of group g of the part
        const auto scale = [&](int i, int g) {
            return as_h2(__byte_perm(s[2 * i][g / 2], s[2 * i + 1][g / 2], g & 1 ? 0x7632 : 0x5410));
        };
        constexpr int BB = (D / 16) / SPLIT;  // runs of sixteen dimensions
#pragma unroll
        for (int n = 0; n < BB; ++n) {
            const int d = 16 * (p.part * BB + n) + 2 * p.r;
            uint32_t even[4], odd[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 sc = scale(i, n / 2);
                if constexpr (BITS == 4) {
                    const uint32_t u =
                        __byte_perm(w[2 * i][n / 4], w[2 * i + 1][n / 4], n & 2 ? 0x7632 : 0x5410) >> (8 * (n & 1));
                    even[i] = h2_bits(__hmul2(__hsub2(as_h2((u & 0x000F000Fu) | 0x64006400u), __float2half2_rn(1032.0f)), sc));
                    odd[i] = h2_bits(__hmul2(__hfma2(as_h2((u & 0x00F000F0u) | 0x64006400u), __float2half2_rn(0.0625f),
                                                     __float2half2_rn(-72.0f)), sc));
                } else {
                    // bytes 2n, 2n + 1 of both tokens under 0x64
                    const uint32_t u = __byte_perm(w[2 * i][n / 2], w[2 * i + 1][n / 2], n & 1 ? 0x7632 : 0x5410);
                    const __half2 z = __float2half2_rn(1152.0f);
                    even[i] = h2_bits(__hmul2(__hsub2(as_h2((u & 0x00FF00FFu) | 0x64006400u), z), sc));
                    odd[i] = h2_bits(__hmul2(__hsub2(as_h2((u >> 8 & 0x00FF00FFu) | 0x64006400u), z), sc));
                }
            }
            put(d, even);
            put(d + 1, odd);
        }
    }
    // The slow way: NaN scales are taken out and their groups noted, large tokens taken down.
    // Returns a bit each of the warp's 32 tokens that are, and in the high word whether
    // there was a NaN.
    __device__ __forceinline__ uint64_t tame(const TokenRows &rows, int t0, uint8_t *nan_groups, const Place &p) {
        uint32_t all = 0u, big = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t groups = 0u;
#pragma unroll
            for (int k = 0; k < SW; ++k) {
                const uint32_t nan = __vcmpgtu2(s[i][k] & 0x7FFF7FFFu, 0x7C007C00u);
                groups |= (nan & 1u) << (2 * k) | (nan >> 16 & 1u) << (2 * k + 1);
                s[i][k] &= ~nan;
            }
            all |= groups;
            bool down = Big<BITS>::some(s[i]);
            if constexpr (SPLIT == 2) {  // one power serves a token's whole row
                uint32_t o[SW] = {};
                const int t = t0 + 8 * p.chunk + i;
                const int64_t r = rows.seen(t) ? rows.row(t, 1) : -1;
                if (r >= 0) load_global<SW>(o, rows.cache.scales + r * F::kGroups + (1 - p.part) * SW * 2);
                down |= Big<BITS>::some(o);
            }
            if (down) {
                Big<BITS>::down(s[i]);
                big |= 1u << (8 * (p.chunk & 3) + i);
            }
            // every run of a row notes the same groups; the parts of a row their own
            if (p.r == 0) nan_groups[p.part * BN + 8 * p.chunk + i] = static_cast<uint8_t>(groups << (p.part * 2 * SW));
        }
        big = __reduce_or_sync(0xffffffffu, big);
        return static_cast<uint64_t>(__any_sync(0xffffffffu, all != 0u)) << 32 | big;
    }
};

// ---- the kernel ------------------------------------------------------------------------------

template <int D, int BITS, int QT>
__global__ void __launch_bounds__(WideShape<D, BITS, QT>::kThreads, 1) kv_attention_wide_kernel(const KvAttnArgs a) {
    using S = WideShape<D, BITS, QT>;
    using L = typename S::L;
    constexpr int BN = S::BN, NQ = S::NQ;
    extern __shared__ uint8_t wide_raw[];
    __shared__ WideShared sh;
    __shared__ uint8_t nan_groups[2][2 * BN];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *qs = wide_raw + ((1024u - (smem_addr(wide_raw) & 1023u)) & 1023u);
    uint8_t *ks = qs + QT * S::kQuery, *vs = ks + S::kKeyStages * S::kKeyStage;

    pdl_trigger();
    pdl_wait();
    Line line = {};
    Cut<L> cut(1, 1);
    int own_head = 0;  // of the CTA's only (query tile, head), where it has just one
    if (a.direct) {
        line.item = blockIdx.x / static_cast<uint32_t>(a.cache.Hkv);
        own_head = static_cast<int>(blockIdx.x - static_cast<uint32_t>(line.item) * static_cast<uint32_t>(a.cache.Hkv));
        const Item<L> it = make_item<L>(a, line.item);
        if (it.bad && own_head == 0 && threadIdx.x == 0) atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
        if (it.n == 0) {
            store_zeros<D, L, S::kThreads>(a, it, own_head);
            return;
        }
    } else {
        line = find_unit<L, S::kThreads>(a, blockIdx.x == 0, sh.scratch);
        store_empty<D, L, S::kThreads>(a);
        cut = Cut<L>(line.units, a.grid);
        if (line.units == 0 || blockIdx.x >= cut.ctas) return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 128);
            mbar_init(&sh.k_full[i], 128);
            mbar_init(&sh.v_full[i], 128);
            mbar_init(&sh.p_full[i], 128);
            mbar_init(&sh.k_free[i], 1);
            mbar_init(&sh.v_free[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init(&sh.drained, 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == S::kWarps - 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    // Every role walks the CTA's runs in the same order; n counts its tiles over all.
    const auto each_run = [&](auto &&body) {
        walk_runs<S::kSlot>(a, cut, blockIdx.x, line.item, line.before, own_head, threadIdx.x == 0, body);
    };

    if (warp < 4 * QT) {
        // -- softmax: one accumulator row a thread -------------------------------------------
        const uint32_t qt = warp >> 2;
        const int row = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t obase = tmem + lanes + S::kO + qt * D;
        uint8_t *const qtile = qs + qt * S::kQuery;
        uint32_t n = 0, c = 0;  // tiles so far: of the CTA, and those this query tile took
        each_run([&](const Item<L> &it, int head, int k0, int k1, float *part) {
            const int col = static_cast<int>(qt) * 128 + row;
            if (static_cast<int>(qt) * 128 >= it.ncols) {  // no columns for this query tile
                n += k1 - k0;
                return true;
            }
            const bool live = col < it.ncols;
            const int f = it.f0 + (live ? col : 0);
            const int pos = live ? it.pos0 + f / a.group : -1;
            float factor;
            {
                // the query, scaled by a power of two so that its largest element lies in
                // [2^13, 2^14), and with the scale's sign
                const uint16_t *src = a.q + (it.row0 + f / a.group) * a.q_stride +
                                      (static_cast<int64_t>(head) * a.group + f % a.group) * D;
                uint32_t top = 0u;
                if (pos >= 0) {  // (a query that sees no token counts as zeros)
#pragma unroll 8
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 v = ld_ro16(src + 8 * i);
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
                    }
                }
                const uint32_t amax = max(top & 0xFFFFu, top >> 16);
                const bool finite = amax < 0x7F80u;
                int e = static_cast<int>(amax >> 7);
                e = e < 14 ? 14 : e;
                const float up = copysignf(__uint_as_float(static_cast<uint32_t>(267 - (finite ? e : 127)) << 23),
                                           a.scale_log2);
                factor = fmaxf(ldexpf(fabsf(a.scale_log2), e - 140), 0x1p-126f);
                if (!finite) factor = __uint_as_float(0x7FC00000u);
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = pos >= 0 && finite ? ld_ro16(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
                    const float x[8] = {bf_lo(v.x) * up, bf_hi(v.x) * up, bf_lo(v.y) * up, bf_hi(v.y) * up,
                                        bf_lo(v.z) * up, bf_hi(v.z) * up, bf_lo(v.w) * up, bf_hi(v.w) * up};
                    uint4 o;
                    if constexpr (BITS == 4)
                        o = make_uint4(h2_bits(__floats2half2_rn(x[0], x[4])), h2_bits(__floats2half2_rn(x[1], x[5])),
                                       h2_bits(__floats2half2_rn(x[2], x[6])), h2_bits(__floats2half2_rn(x[3], x[7])));
                    else
                        o = make_uint4(h2_bits(__floats2half2_rn(x[0], x[1])), h2_bits(__floats2half2_rn(x[2], x[3])),
                                       h2_bits(__floats2half2_rn(x[4], x[5])), h2_bits(__floats2half2_rn(x[6], x[7])));
                    *reinterpret_cast<uint4 *>(qtile + (i >> 3) * (128 * 128) + row * 128 +
                                               (((i & 7) ^ (row & 7)) << 4)) = o;
                }
            }
            fence_async_shared();
            mbar_arrive(&sh.q_full[qt]);

            float m = -INFINITY, ref = 0.0f, l = 0.0f;
            uint32_t nan_mask = 0u;  // groups of which a visible value is NaN
            // first visible token of the window (sinks apart), for the masked tiles
            const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
            // Multiplies O and the weights of the tile's first `chunks` quarters by scale.
            const auto rescale = [&](bool sums, int chunks, float scale, uint32_t sbase) {
                if (chunks) scale_weights(sbase, chunks, scale);
                if (!sums) return true;
                if (!wide_wait_warp(sh, &sh.pv_done[S::buf(qt, c - 1)], S::phase(c - 1))) return false;
                tc_fence_after();
#pragma unroll 1
                for (int i = 0; i < D; i += 16) {
                    uint32_t x[16];
                    tmem_load16(x, obase + i);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * scale);
                    tmem_store16(obase + i, x);
                }
                tmem_wait_store();
                return true;
            };
            for (int k = k0; k < k1; ++k, ++n, ++c) {
                const uint32_t b = S::buf(qt, c), vstage = S::stage(n);
                const int t0 = it.token(k);
                if (!wide_wait_warp(sh, &sh.s_full[b], S::phase(c))) return false;
                tc_fence_after();
                const uint32_t sbase = tmem + lanes + b * BN;
                const bool masked = t0 + BN - 1 > it.lo_pos ||
                                    (a.window && t0 <= it.hi - 1 - a.window && t0 + BN > a.sinks);
                // bit j: the row does not see token t0 + 32i + j
                const auto hidden = [&](int i) { return hidden_tokens(pos, lo, a.sinks, t0 + 32 * i); };
                // (the values' flags are there once their stage is)
                if (!wide_wait_warp(sh, &sh.v_full[vstage], S::round(n))) return false;
                const uint32_t vflags = sh.val_flags[vstage];
                if ((sh.key_flags[n & 7] | vflags) & 0x01010101u) {
                    const float large = large_logits<BN, Big<BITS>::kDown>(sbase, sh.key_big[n & 7], sh.val_big[vstage],
                                                                           factor, pos, lo, a.sinks, t0);
                    sh.large[threadIdx.x] = large;
                    if (large > m && m != -INFINITY) m = -FLT_MAX;  // the first chunk seen takes a new reference
                }
#pragma unroll 1
                for (int i = 0; i < BN / 32; ++i) {
                    uint32_t v[32];
                    tmem_load32(v, sbase + 32 * i);
                    const uint32_t mask = masked ? hidden(i) : 0u;
                    tmem_wait_load(v);
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (mask >> j & 1u) v[j] = 0xFF800000u;
                    }
                    float most = __uint_as_float(v[0]);
#pragma unroll
                    for (int j = 1; j < 31; j += 2)
                        most = max3(most, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                    const float top = fmaxf(most, __uint_as_float(v[31])) * factor;
                    if (__any_sync(0xffffffffu, top > m)) {
                        // References are whole numbers, so a rescale is exact: of O, and of
                        // this tile's weights already stored.
                        float scale = 1.0f;
                        if (top > m) {
                            const float least = vflags & 0x01010101u ? fmaxf(top, sh.large[threadIdx.x]) : top;
                            const float nref = ceilf(least) + (kWideSlack - kWideRoom);
                            if (m != -INFINITY) scale = exp2_approx(ref - nref);
                            ref = nref;
                            m = nref + kWideRoom;
                            l *= scale;
                        }
                        __syncwarp();  // (tensor memory is for whole warps)
                        if (!rescale(k > k0, i, scale, sbase)) return false;
                    }
                    const float shift = -ref;
                    uint32_t y[16];
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float p0, p1;
                        fma2(p0, p1, __uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]), factor, shift);
                        p0 = exp2_approx(p0);
                        p1 = exp2_approx(p1);
                        add_pairs(sum[0], sum[1], p0, p1);
                        y[j] = h2_bits(__floats2half2_rn(p0, p1));
                    }
                    tmem_store16(sbase + 16 * i, y);  // over columns already read
                    l += sum[0] + sum[1];
                }
                if (vflags) {
                    if (vflags & 0x01010101u) large_weights<BN, Big<BITS>::kDown>(sbase, sh.val_big[vstage]);
                    for (int w = 0; w < 4; ++w) {
                        if (!(vflags >> (8 * w) & 2u)) continue;
                        const int first = BN == 64 ? 32 * (w & 1) : 32 * w, part_of = BN == 64 ? BN * (w >> 1) : 0;
                        const uint32_t mask = hidden(first / 32);
                        for (int j = 0; j < 32; ++j)
                            if (!(mask >> j & 1u)) nan_mask |= nan_groups[vstage][part_of + first + j];
                    }
                }
                tmem_wait_store();
                tc_fence_before();
                mbar_arrive(&sh.p_full[b]);
            }
            // -- the run's sums: finished, or a piece ---------------------------------------
            if (!wide_wait_warp(sh, &sh.pv_done[S::buf(qt, c - 1)], S::phase(c - 1))) return false;
            tc_fence_after();
            const int64_t out_row = (it.row0 + f / a.group) * a.Hq + static_cast<int64_t>(head) * a.group + f % a.group;
            // (a piece carries the 2^-24 that the other kernel's sums have)
            const float scale = part ? 0x1p-24f : (l == 0.0f ? 0.0f : 1.0f / l);
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
                uint32_t x[32];
                tmem_load32(x, obase + 32 * i);
                tmem_wait_load(x);
                const float unit = nan_mask >> i & 1u ? __uint_as_float(0x7FC00000u) : scale;
                float y[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(x[j]) * unit;
                if (live && part) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4 *>(part + col * D + 32 * i + j) =
                            make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                } else if (live) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
                        st16(a.out + out_row * D + 32 * i + j,
                             make_uint4(pack_bf2(y[j], y[j + 1]), pack_bf2(y[j + 2], y[j + 3]),
                                        pack_bf2(y[j + 4], y[j + 5]), pack_bf2(y[j + 6], y[j + 7])));
                }
                __syncwarp();  // (the next load is the whole warp's)
            }
            if (live && part) {
                part[NQ * D + col] = m == -INFINITY ? -INFINITY : ref;
                part[NQ * D + NQ + col] = l;
            } else if (live && a.lse) {
                a.lse[out_row] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
            }
            tc_fence_before();  // O is read before the next run's products
            return true;
        });
    } else if (warp < 4 * QT + 4) {
        // -- keys -----------------------------------------------------------------------------
        const int w = warp - 4 * QT;
        uint32_t n = 0;
        each_run([&](const Item<L> &it, int head, int k0, int k1, float *) {
            const TokenRows rows(a, it, head);
            KeyTile<D, BITS, BN> tile;
            tile.load(rows, it.token(k0), w, lane);
            for (int k = k0; k < k1; ++k, ++n) {
                const uint32_t s = S::key_stage(n), par = S::key_round(n);
                // the products that read this stage before are over
                if (!wide_wait_warp(sh, &sh.k_free[s], par ^ 1)) return false;
                uint32_t big = 0u;
                if (__any_sync(0xffffffffu, tile.special()))
                    big = tile.tame(lane);
                tile.store(ks + s * S::kKeyStage, w, lane);
                if (lane == 0) {
                    reinterpret_cast<uint8_t *>(&sh.key_flags[n & 7])[w] = big ? 1 : 0;
                    if constexpr (BN == 128)
                        sh.key_big[n & 7][w] = big;
                    else
                        reinterpret_cast<uint16_t *>(sh.key_big[n & 7])[w] = static_cast<uint16_t>(big);
                }
                fence_async_shared();
                mbar_arrive(&sh.k_full[s]);
                // the next tile's bytes come while this one is used
                if (k + 1 < k1) tile.load(rows, it.token(k + 1), w, lane);
            }
            return true;
        });
    } else if (warp < 4 * QT + 8) {
        // -- values ---------------------------------------------------------------------------
        const int w = warp - 4 * QT - 4;
        const auto place = ValueTile<D, BITS, BN>::place(w, lane);
        uint32_t n = 0;
        each_run([&](const Item<L> &it, int head, int k0, int k1, float *) {
            const TokenRows rows(a, it, head);
            ValueTile<D, BITS, BN> tile;
            tile.load(rows, it.token(k0), place);
            for (int k = k0; k < k1; ++k, ++n) {
                const uint32_t s = S::stage(n), par = S::round(n);
                if (!wide_wait_warp(sh, &sh.v_free[s], par ^ 1)) return false;
                uint64_t met = 0u;
                if (__any_sync(0xffffffffu, tile.special()))
                    met = tile.tame(rows, it.token(k), nan_groups[s], place);
                tile.store(vs + s * S::kStage, place);
                if (lane == 0) {
                    const uint32_t big = static_cast<uint32_t>(met);
                    sh.val_big[s][w] = big;  // (of 64 tokens, twice)
                    reinterpret_cast<uint8_t *>(&sh.val_flags[s])[w] = (big ? 1 : 0) | (met >> 32 ? 2 : 0);
                }
                fence_async_shared();
                mbar_arrive(&sh.v_full[s]);
                if (k + 1 < k1) tile.load(rows, it.token(k + 1), place);
            }
            return true;
        });
    } else if (lane == 0) {
        // -- products ---------------------------------------------------------------------------
        const uint32_t qa = smem_addr(qs), ka = smem_addr(ks), va = smem_addr(vs);
        uint32_t n = 0, runs[2] = {0, 0}, s_done[2] = {0, 0}, pv_count[2] = {0, 0};
        // S of query tile qt with the keys of the CTA's tile i, into the buffer of the
        // query tile's next tile: its weights of before have been used up
        const auto logits = [&](uint32_t qt, uint32_t i, bool last) {
            const uint32_t c = s_done[qt]++, b = S::buf(qt, c), s = S::key_stage(i);
            constexpr uint32_t kBack = S::kBufs;
            if (c >= kBack && !wide_wait(sh, &sh.pv_done[b], S::phase(c - kBack))) return false;
            if (!wide_wait(sh, &sh.k_full[s], S::key_round(i))) return false;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < D / 16; ++q)
#pragma unroll
                for (int rest = 0; rest < 2; ++rest)
                    mma_ss(tmem + b * BN, operand_desc(qa + qt * S::kQuery + (q >> 2) * (128 * 128) + (q & 3) * 32),
                           operand_desc(ka + s * S::kKeyStage + rest * S::kStage + (q >> 2) * (BN * 128) + (q & 3) * 32),
                           wide_idesc(BN), q != 0 || rest != 0);
            tc_commit(&sh.s_full[b]);
            if (last) tc_commit(&sh.k_free[s]);
            return true;
        };
        const auto outputs = [&](uint32_t qt, uint32_t i, bool first, bool last) {
            const uint32_t c = pv_count[qt]++, b = S::buf(qt, c), s = S::stage(i);
            if (!wide_wait(sh, &sh.p_full[b], S::phase(c)) || !wide_wait(sh, &sh.v_full[s], S::round(i))) return false;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < BN / 16; ++q)
                mma_ts(tmem + S::kO + qt * D, tmem + b * BN + 8 * q,
                       operand_desc(va + s * S::kStage + (q >> 2) * (D * 128) + (q & 3) * 32), wide_idesc(D),
                       !(first && q == 0));
            tc_commit(&sh.pv_done[b]);
            if (last) tc_commit(&sh.v_free[s]);
            return true;
        };
        each_run([&](const Item<L> &it, int, int k0, int k1, float *) {
            const uint32_t tiles = it.ncols > 128 ? 2 : 1, end = n + (k1 - k0), start = n;
            for (uint32_t qt = 0; qt < tiles; ++qt) {
                if (!wide_wait(sh, &sh.q_full[qt], runs[qt] & 1)) return false;
                ++runs[qt];
            }
            for (uint32_t qt = 0; qt < tiles; ++qt)
                if (!logits(qt, n, qt + 1 == tiles)) return false;
            for (; n < end; ++n) {
                for (uint32_t qt = 0; qt < tiles; ++qt) {
                    // with a second buffer the next logits come first, beside this softmax
                    if (S::kBufs == 2 && n + 1 < end && !logits(qt, n + 1, qt + 1 == tiles)) return false;
                    if (!outputs(qt, n, n == start, qt + 1 == tiles)) return false;
                    if (S::kBufs == 1 && n + 1 < end && !logits(qt, n + 1, qt + 1 == tiles)) return false;
                }
            }
            return true;
        });
        // nothing of this CTA is under way any more when its tensor memory goes back
        tc_commit(&sh.drained);
        if (!mbar_wait_bounded(&sh.drained, 0, 2000000000ull, nullptr))
            atomicOr(&g_kv_attention_status, RN_STATUS_WAIT_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == S::kWarps - 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

int kv_attention_wide_status(unsigned int *out, int clear) {
    return kv_status_word(g_kv_attention_status, out, clear);
}

// ---- host --------------------------------------------------------------------------------------

template <int D, int BITS, int QT>
static int wide_launch_of(KvAttnArgs &a, cudaStream_t st) {
    using S = WideShape<D, BITS, QT>;
    // A CTA for each (query tile, head), without line and joining, where there are few
    // tiles of tokens, or heads to fill the GPU with them, or so many that the last round
    // does not matter (chunks of a quarter of their context, 8 heads of 128, us on the
    // line / directly: contexts of 600, 1 sequence 32 / 33, 32 of them 204 / 175; 2000, 1
    // sequence 62 / 72, 8 of them 298 / 272; 3000, 16 of them 1089 / 1030).
    const int64_t most = attn_most_tokens(a, S::NQ), busy = attn_busy_heads(a, S::NQ);
    a.direct = a.heads <= 2 * busy && a.heads <= INT32_MAX &&  // few CTAs without work
               (most <= 640 || (most <= 2048 && 5 * busy >= 3 * static_cast<int64_t>(a.grid)) ||
                busy >= 4 * static_cast<int64_t>(a.grid));
    static std::atomic<int> attr_done[kMaxDevices];
    const int dev = current_device_index();
    if (dev < 0 || dev >= kMaxDevices) return RN_ERR_DEVICE;
    const auto kernel = kv_attention_wide_kernel<D, BITS, QT>;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess) {
            cudaGetLastError();
            return RN_ERR_DEVICE;
        }
        attr_done[dev].store(1, std::memory_order_release);
    }
    const unsigned ctas = static_cast<unsigned>(a.direct ? a.heads : a.grid);
    const int rc = launch_pdl(kernel, dim3(ctas), dim3(S::kThreads), S::kSmem, st, a);
    if (rc != RN_OK || a.direct) return rc;
    return join_launch<D, typename S::L>(a, st);
}

static int query_tiles(int D, int64_t columns) { return D <= 128 && columns > 128 ? 2 : 1; }

AttnPlan wide_plan(int sm_count, int64_t B, int group, int D, int64_t max_q_len) {
    const int64_t nq = 128 * query_tiles(D, max_q_len * group);
    AttnPlan p;
    p.q_tiles = (max_q_len * group + nq - 1) / nq;
    p.grid = sm_count;
    p.head_bytes = 16 + 32 * static_cast<int64_t>(p.grid);
    p.bytes = p.head_bytes + static_cast<int64_t>(p.grid) * 2 * nq * (D + 2) * 4;
    return p;
}

int wide_launch(int D, int format, KvAttnArgs &a, cudaStream_t st) {
    const int tiles = query_tiles(D, a.max_q_len * a.group);
    return kv_dispatch(D, format, [&](auto d, auto bits) {
        if constexpr (d.value <= 128)
            if (tiles == 2) return wide_launch_of<d.value, bits.value, 2>(a, st);
        return wide_launch_of<d.value, bits.value, 1>(a, st);
    });
}

}  // namespace rn
