// kv_attention_wide.cu -- attention of many queries a sequence over the quantised
// key/value cache (sm_103a): chunks of a prompt against what the cache holds.
//
// The same formula as kv_attention.cu with 128 columns (queries times heads of the
// group) at a time, which makes it a matter of arithmetic: 4 D flops for each
// column and token against one restored key and value.  The products run as
// tcgen05.mma with the columns as the 128 rows of the accumulator:
//   S = Q K'^T    Q and K' in shared memory, S in tensor memory,
//   O += P V'     P in tensor memory (over its S), V' in shared memory.
// K' and V' are the cached values restored to fp16, s * c rounded once (2^-11);
// both operands of S are exact otherwise, the queries as in kv_attention.cu.  A
// tile with a scale above 255 is restored at 2^-8 of its size (the weights, or
// the logit's factor, make up for it), so nothing leaves fp16.
//
// Roles: warps 0-3 one accumulator row a thread (softmax, output), warps 4-7
// restore keys, 8-11 values (two stages each), one thread of warp 12 issues the
// products.  S has two buffers, so the product of tile n + 1 runs beside the
// softmax of tile n.  What bounds it: the exponentials (16 a clock and SM) and the
// tensor cores need about 1000 clocks a tile of 128 x 128 x 128 each, shared memory
// traffic 1300 (192 KB: the operands once, K' and V' written).
//
// Shared memory operands are K-major with the 128-byte exchange of 16-byte chunks
// (chunk ^ row % 8 in rows of 128 bytes): 64 elements a row, blocks of 64 elements
// one after the other.  In 4 bits the eight dimensions of a chunk lie in the order
// 0 4 1 5 2 6 3 7, the order in which they leave a word, in Q as in K'.
#include "kv_attention.cuh"

namespace rn {

constexpr int kWideWarps = 13;
constexpr int kWideThreads = 32 * kWideWarps;
constexpr float kWideRoom = 6.0f;   // weights stay below 2^6 (2^14 where values are at 2^-8)
constexpr float kWideSlack = 4.0f;  // powers of two a weight may grow before a rescale
constexpr uint64_t kWideTimeout = 2000000000ull;

template <int D, int BITS>
struct WideShape {
    using F = KvFormat<D, BITS>;
    static constexpr int BN = D == 256 ? 64 : 128;  // tokens of a tile
    using L = LineShape<128, BN, 4, 1>;
    static constexpr int kQuery = 128 * D * 2;
    static constexpr int kStage = BN * D * 2;        // a tile's keys, or values
    static constexpr int kUsed = 1024 + kQuery + 4 * kStage;
    // more than half of an SM's shared memory: the tensor memory of an SM has one owner
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static constexpr int kSlot = 128 * (D + 2);
    static constexpr uint32_t kO = 2 * BN;           // tensor memory columns: S0, S1, O
    static_assert(kO + D <= 512, "tensor memory");
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
// 32 columns of the warp's 32 rows, one row a thread; complete on return.
__device__ __forceinline__ void tmem_load32(float (&r)[32], uint32_t addr) {
    uint32_t u[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
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

constexpr uint32_t kScale255 = 0x5BF8u;  // fp16 255: larger scales (and NaN) take the slow way

struct WideShared {
    uint64_t q_full, k_full[2], v_full[2], s_full[2], p_full[2], pv_done[2], drained;
    uint32_t tmem;
    int abort;
    // powers of two taken off, by restoring warp: keys of four tiles (their producer runs
    // ahead of the softmax by up to three), values of two
    int key_exp[4][4], val_exp[2][4], val_nan[2][4];
    int64_t scratch[kWideWarps + 2];
};

// A wait with a limit; gives up for the whole CTA when it runs out.
__device__ __forceinline__ bool wide_wait(WideShared &sh, uint64_t *bar, uint32_t parity) {
    if (mbar_wait_bounded(bar, parity, kWideTimeout, &sh.abort)) return true;
    if (atomicExch(&sh.abort, 1) == 0) atomicOr(&g_kv_attention_status, RN_STATUS_WAIT_TIMEOUT);
    return false;
}
// The same by a whole warp, which is together again afterwards.
__device__ __forceinline__ bool wide_wait_warp(WideShared &sh, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wide_wait(sh, bar, parity));
}

// What a thread needs to find a token's rows.
template <int D, int BITS, class L>
struct TokenRows {
    const KvAttnArgs &a;
    const Item<L> &it;
    int kvh;

    __device__ __forceinline__ bool seen(int t) const {
        return t < it.hi && (it.win_lo == 0 || t < a.sinks || t >= it.win_lo);
    }
    // The row of token t's key (which 0) or value, or -1: nothing of t .. t + n - 1 is
    // seen (n tokens of one page), or its page does not exist.
    __device__ __forceinline__ int64_t row(int t, int n, int which) const {
        bool any = false;
        for (int i = 0; i < n; ++i) any |= seen(t + i);
        if (!any) return -1;
        const int page = a.page_table[it.seq * a.max_pages + (t >> a.cache.log2_page)];
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.cache.num_pages)) {
            atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
            return -1;
        }
        return a.cache.row(page, which, kvh, t & ((1 << a.cache.log2_page) - 1));
    }
};

// ---- restoring keys ---------------------------------------------------------------------
// Four warps, BN / 4 tokens each (each with a power of two of its own), eight at a time: lane = token % 8 + 8 j with j the
// quarter of the stored row.  A group's eight elements are one chunk of the operand.
template <int D, int BITS>
struct KeyTile {
    using S = WideShape<D, BITS>;
    using F = KvFormat<D, BITS>;
    static constexpr int ITER = S::BN / 32, KW = F::kGroups * BITS / 4, SW = F::kGroups / 2;
    uint32_t w[ITER][KW], s[ITER][SW];

    template <class Rows>
    __device__ __forceinline__ void load(const Rows &rows, int t0, int warp, int lane) {
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int64_t r = rows.row(t0 + warp * (S::BN / 4) + 8 * i + (lane & 7), 1, 0);
            if (r >= 0) {
                load_global<KW>(w[i], rows.a.cache.codes + r * F::kRow + (lane >> 3) * KW * 4);
                load_global<SW>(s[i], rows.a.cache.scales + r * F::kGroups);
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
        return max(m & 0xFFFFu, m >> 16) > kScale255;
    }
    __device__ __forceinline__ void store(uint8_t *stage, int warp, int lane, bool small) const {
        const __half2 down = __float2half2_rn(small ? 0.00390625f : 1.0f);
#pragma unroll
        for (int i = 0; i < ITER; ++i) {
            const int row = warp * (S::BN / 4) + 8 * i + (lane & 7);
#pragma unroll
            for (int g = 0; g < F::kGroups; ++g) {
                const __half2 pair = as_h2(s[i][g / 2]);
                const __half2 sc = __hmul2(g & 1 ? __high2half2(pair) : __low2half2(pair), down);
                __half2 h[4];
                if constexpr (BITS == 4)
                    codes_of(w[i][g], h);
                else
                    codes_of(w[i][2 * g], w[i][2 * g + 1], h);
                const int chunk = 4 * g + (lane >> 3);
                *reinterpret_cast<uint4 *>(stage + (chunk >> 3) * (S::BN * 128) + row * 128 +
                                           (((chunk & 7) ^ (row & 7)) << 4)) =
                    make_uint4(h2_bits(__hmul2(h[0], sc)), h2_bits(__hmul2(h[1], sc)), h2_bits(__hmul2(h[2], sc)),
                               h2_bits(__hmul2(h[3], sc)));
            }
        }
    }
};

// ---- restoring values, transposed --------------------------------------------------------
// A thread takes eight tokens of the stored rows' r-th run (or half of it, D 256) and
// writes, for each of its dimensions, the eight tokens as one chunk of that
// dimension's row.  r and the tokens are mixed over the lanes so that eight
// neighbours write eight different banks' chunks.
template <int D, int BITS>
struct ValueTile {
    using S = WideShape<D, BITS>;
    using F = KvFormat<D, BITS>;
    static constexpr int SPLIT = D == 256 ? 2 : 1;
    static constexpr int VW = D * BITS / 256 / SPLIT, SW = BITS == 4 ? VW : (VW + 1) / 2;
    uint32_t w[8][VW], s[8][SW];
    uint32_t other;  // D 256: the largest scales of the row's other part

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
    template <class Rows>
    __device__ __forceinline__ void load(const Rows &rows, int t0, const Place &p) {
        const int t = t0 + 8 * p.chunk;
        const int64_t r = rows.row(t, 8, 1);
        other = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r >= 0 && rows.seen(t + i)) {
                load_global<VW>(w[i], rows.a.cache.codes + (r + i) * F::kRow + (p.r * SPLIT + p.part) * VW * 4);
                load_global<SW>(s[i], rows.a.cache.scales + (r + i) * F::kGroups + p.part * SW * 2);
                if constexpr (SPLIT == 2) {
                    // one exponent serves a token's whole row
                    uint32_t o[SW];
                    load_global<SW>(o, rows.a.cache.scales + (r + i) * F::kGroups + (1 - p.part) * SW * 2);
#pragma unroll
                    for (int k = 0; k < SW; ++k) other = __vmaxu2(other, o[k]);
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
        return max(m & 0xFFFFu, m >> 16) > kScale255;
    }
    // The slow way: scales at 2^-8, NaN scales taken out and their groups noted.
    __device__ __forceinline__ bool tame(uint8_t *nan_groups, const Place &p) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t groups = 0u;
#pragma unroll
            for (int k = 0; k < SW; ++k) {
                uint32_t lo = s[i][k] & 0xFFFFu, hi = s[i][k] >> 16;
                if ((lo & 0x7FFFu) > 0x7C00u) {
                    lo = 0u;
                    groups |= 1u << (2 * k);
                }
                if ((hi & 0x7FFFu) > 0x7C00u) {
                    hi = 0u;
                    groups |= 2u << (2 * k);
                }
                s[i][k] = h2_bits(__hmul2(as_h2(lo | hi << 16), __float2half2_rn(0.00390625f)));
            }
            any |= groups != 0u;
            // every run of a row notes the same groups; the parts of a row their own
            if (p.r == 0) nan_groups[(p.part * S::BN) + 8 * p.chunk + i] = static_cast<uint8_t>(groups << (p.part * 2 * SW));
        }
        return any;
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
};

// ---- the kernel ------------------------------------------------------------------------------

template <int D, int BITS>
__global__ void __launch_bounds__(kWideThreads, 1) kv_attention_wide_kernel(const KvAttnArgs a) {
    using S = WideShape<D, BITS>;
    using F = KvFormat<D, BITS>;
    using L = typename S::L;
    constexpr int BN = S::BN;
    extern __shared__ uint8_t wide_raw[];
    __shared__ WideShared sh;
    __shared__ uint8_t nan_groups[2][2 * BN];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *qs = wide_raw + ((1024u - (smem_addr(wide_raw) & 1023u)) & 1023u);
    uint8_t *ks = qs + S::kQuery, *vs = ks + 2 * S::kStage;

    pdl_trigger();
    pdl_wait();
    const Line line = find_unit<L, kWideThreads>(a, blockIdx.x == 0, sh.scratch);
    const Cut<L> cut(line.units, a.grid);
    if (line.units == 0 || blockIdx.x >= cut.ctas) return;
    if (threadIdx.x == 0) {
        mbar_init(&sh.q_full, 128);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.k_full[i], 128);
            mbar_init(&sh.v_full[i], 128);
            mbar_init(&sh.p_full[i], 128);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init(&sh.drained, 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    // Every role walks the CTA's runs in the same order; n counts its tiles over all.
    const int64_t u0 = cut.start(blockIdx.x), u1 = cut.start(blockIdx.x + 1);
    const auto each_run = [&](auto &&body) {
        int64_t item = line.item, before = line.before, u = u0;
        while (u < u1) {
            const Item<L> it = make_item<L>(a, item);
            if (it.n == 0) {
                ++item;
                continue;
            }
            const int units = it.units();
            const int64_t in = u - before * a.cache.Hkv;
            const int head = static_cast<int>(quotient(in, units));
            const int v0 = static_cast<int>(in - static_cast<int64_t>(head) * units);
            const int64_t left = u1 - u;
            const int v1 = units - v0 <= left ? units : v0 + static_cast<int>(left);
            const int k0 = v0 > L::LEAD ? v0 - L::LEAD : 0, k1 = v1 - L::LEAD;
            if (k1 > k0) {
                float *part = nullptr;
                if (k1 - k0 != it.n)
                    part = a.partial + (2 * static_cast<int64_t>(blockIdx.x) + (u == u0 ? 0 : 1)) * S::kSlot;
                if (!body(it, head, k0, k1, part)) return;
            }
            u += v1 - v0;
            if (v1 == units && head == a.cache.Hkv - 1) {
                before += units;
                ++item;
            }
        }
    };

    uint32_t n = 0;  // tiles so far
    if (warp < 4) {
        // -- softmax: one accumulator row a thread -------------------------------------------
        const int row = threadIdx.x;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        each_run([&](const Item<L> &it, int head, int k0, int k1, float *part) {
            const bool live = row < it.ncols;
            const int f = it.f0 + (live ? row : 0);
            const int pos = live ? it.pos0 + f / a.group : -1;
            float factor;
            {
                // the query, scaled by a power of two so that its largest element lies in
                // [2^13, 2^14), and with the scale's sign
                const uint16_t *src = a.q + (it.row0 + f / a.group) * a.q_stride +
                                      (static_cast<int64_t>(head) * a.group + f % a.group) * D;
                uint32_t top = 0u;
                if (live)
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 v = ld_ro16(src + 8 * c);
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
                    }
                const uint32_t amax = max(top & 0xFFFFu, top >> 16);
                const bool finite = amax < 0x7F80u;
                int e = static_cast<int>(amax >> 7);
                e = e < 14 ? 14 : e;
                const float up = copysignf(__uint_as_float(static_cast<uint32_t>(267 - (finite ? e : 127)) << 23),
                                           a.scale_log2);
                factor = fmaxf(ldexpf(fabsf(a.scale_log2), e - 140), 0x1p-126f);
                if (!finite) factor = __uint_as_float(0x7FC00000u);
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = live && finite ? ld_ro16(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
                    const float x[8] = {bf_lo(v.x) * up, bf_hi(v.x) * up, bf_lo(v.y) * up, bf_hi(v.y) * up,
                                        bf_lo(v.z) * up, bf_hi(v.z) * up, bf_lo(v.w) * up, bf_hi(v.w) * up};
                    uint4 o;
                    if constexpr (BITS == 4)
                        o = make_uint4(h2_bits(__floats2half2_rn(x[0], x[4])), h2_bits(__floats2half2_rn(x[1], x[5])),
                                       h2_bits(__floats2half2_rn(x[2], x[6])), h2_bits(__floats2half2_rn(x[3], x[7])));
                    else
                        o = make_uint4(h2_bits(__floats2half2_rn(x[0], x[1])), h2_bits(__floats2half2_rn(x[2], x[3])),
                                       h2_bits(__floats2half2_rn(x[4], x[5])), h2_bits(__floats2half2_rn(x[6], x[7])));
                    *reinterpret_cast<uint4 *>(qs + (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = o;
                }
            }
            fence_async_shared();
            mbar_arrive(&sh.q_full);

            float m = -INFINITY, ref = 0.0f, l = 0.0f;
            uint32_t nan_mask = 0u;  // groups of which a visible value is NaN
            for (int k = k0; k < k1; ++k, ++n) {
                const uint32_t s = n & 1, par = (n >> 1) & 1;
                const int t0 = it.token(k);
                if (!wide_wait_warp(sh, &sh.s_full[s], par) || !wide_wait_warp(sh, &sh.v_full[s], par)) return false;
                tc_fence_after();
                const uint32_t sbase = tmem + lanes + s * BN;
                // the factor of columns 32c + 16h ..
                const auto factor_of = [&](int c, int h) {
                    return factor * static_cast<float>(1 << sh.key_exp[n & 3][(32 * c + 16 * h) / (BN / 4)]);
                };
                const bool masked = t0 + BN - 1 > it.lo_pos ||
                                    (a.window && t0 <= it.hi - 1 - a.window && t0 + BN > a.sinks);
                // first visible token of the window (sinks apart), for the masked tiles
                const int lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;
                const auto hidden = [&](int t) { return t > pos || (t < lo && t >= a.sinks); };
                float x[32];
                float top = -INFINITY;
                for (int c = 0; c < BN / 32; ++c) {
                    tmem_load32(x, sbase + 32 * c);
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (hidden(t0 + 32 * c + i)) x[i] = -INFINITY;
                    }
                    float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 32; ++i) most[i / 16] = fmaxf(most[i / 16], x[i]);
                    top = fmaxf(top, fmaxf(most[0] * factor_of(c, 0), most[1] * factor_of(c, 1)));
                }
                if (__any_sync(0xffffffffu, top > m)) {
                    float scale = 1.0f;
                    if (top > m) {
                        const float nref = top + (kWideSlack - kWideRoom);
                        if (m != -INFINITY) scale = exp2_approx(ref - nref);
                        ref = nref;
                        m = top + kWideSlack;
                        l *= scale;
                    }
                    if (k > k0) {
                        if (!wide_wait_warp(sh, &sh.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) return false;
                        tc_fence_after();
                        for (int c = 0; c < D / 32; ++c) {
                            const uint32_t at = tmem + lanes + S::kO + 32 * c;
                            tmem_load32(x, at);
                            uint32_t y[16];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(x[16 * h + i] * scale);
                                tmem_store16(at + 16 * h, y);
                            }
                        }
                        tmem_wait_store();
                    }
                }
                for (int c = 0; c < BN / 32; ++c) {
                    tmem_load32(x, sbase + 32 * c);
                    uint32_t y[16];
                    const float fk[2] = {factor_of(c, 0), factor_of(c, 1)};
                    const int ve = sh.val_exp[s][c];
                    const float shift = static_cast<float>(ve) - ref;
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = exp2_approx(fmaf(x[i], fk[i / 16], shift));
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (hidden(t0 + 32 * c + i)) x[i] = 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        sum += x[2 * i] + x[2 * i + 1];
                        y[i] = h2_bits(__floats2half2_rn(x[2 * i], x[2 * i + 1]));
                    }
                    tmem_store16(sbase + 16 * c, y);  // over columns already read
                    l = fmaf(sum, ve ? 0.00390625f : 1.0f, l);
                }
                for (int w = 0; w < 4; ++w)
                    if (sh.val_nan[s][w]) {
                        const int first = D == 256 ? 32 * (w & 1) : 32 * w, part_of = D == 256 ? BN * (w >> 1) : 0;
                        for (int t = first; t < first + 32; ++t)
                            if (!hidden(t0 + t)) nan_mask |= nan_groups[s][part_of + t];
                    }
                tmem_wait_store();
                tc_fence_before();
                mbar_arrive(&sh.p_full[s]);
            }
            // -- the run's sums: finished, or a piece ---------------------------------------
            if (!wide_wait_warp(sh, &sh.pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1)) return false;
            tc_fence_after();
            const float top = m == -INFINITY ? -INFINITY : ref;
            for (int c = 0; c < D / 32; ++c) {
                float x[32];
                tmem_load32(x, tmem + lanes + S::kO + 32 * c);
                // store_result undoes 2^-24, which the other kernel's sums carry
                const float unit = nan_mask >> c & 1u ? __uint_as_float(0x7FC00000u) : 0x1p-24f;
                if (live) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 v = make_float4(x[i] * unit, x[i + 1] * unit, x[i + 2] * unit, x[i + 3] * unit);
                        const int d = 32 * c + i;
                        if (part)
                            *reinterpret_cast<float4 *>(part + row * D + d) = v;
                        else
                            store_result<D>(a, it, head * a.group, row, d, v, ref, l);
                    }
                }
            }
            if (part && live) {
                part[128 * D + row] = top;
                part[128 * D + 128 + row] = l;
            }
            tc_fence_before();  // O is read before the next run's products
            return true;
        });
    } else if (warp < 8) {
        // -- keys -----------------------------------------------------------------------------
        const int w = warp - 4;
        each_run([&](const Item<L> &it, int head, int k0, int k1, float *) {
            const TokenRows<D, BITS, L> rows{a, it, head};
            KeyTile<D, BITS> cur, next;
            cur.load(rows, it.token(k0), w, lane);
            for (int k = k0; k < k1; ++k, ++n) {
                const uint32_t s = n & 1, par = (n >> 1) & 1;
                if (k + 1 < k1) next.load(rows, it.token(k + 1), w, lane);
                // the product that read this stage before is over
                if (!wide_wait_warp(sh, &sh.s_full[s], par ^ 1)) return false;
                const bool small = __any_sync(0xffffffffu, cur.special());
                if (lane == 0) sh.key_exp[n & 3][w] = small ? 8 : 0;
                cur.store(ks + s * S::kStage, w, lane, small);
                fence_async_shared();
                mbar_arrive(&sh.k_full[s]);
                cur = next;
            }
            return true;
        });
    } else if (warp < 12) {
        // -- values ---------------------------------------------------------------------------
        const int w = warp - 8;
        const auto place = ValueTile<D, BITS>::place(w, lane);
        each_run([&](const Item<L> &it, int head, int k0, int k1, float *) {
            const TokenRows<D, BITS, L> rows{a, it, head};
            ValueTile<D, BITS> cur, next;
            cur.load(rows, it.token(k0), place);
            for (int k = k0; k < k1; ++k, ++n) {
                const uint32_t s = n & 1, par = (n >> 1) & 1;
                if (k + 1 < k1) next.load(rows, it.token(k + 1), place);
                if (!wide_wait_warp(sh, &sh.pv_done[s], par ^ 1)) return false;
                const bool slow = __any_sync(0xffffffffu, cur.special());
                bool nan = false;
                if (slow) nan = __any_sync(0xffffffffu, cur.tame(nan_groups[s], place));
                if (lane == 0) {
                    sh.val_exp[s][w] = slow ? 8 : 0;
                    sh.val_nan[s][w] = nan;
                }
                cur.store(vs + s * S::kStage, place);
                fence_async_shared();
                mbar_arrive(&sh.v_full[s]);
                cur = next;
            }
            return true;
        });
    } else if (lane == 0) {
        // -- products ---------------------------------------------------------------------------
        const uint32_t qa = smem_addr(qs), ka = smem_addr(ks), va = smem_addr(vs);
        uint32_t run = 0;
        const auto value_product = [&](uint32_t i, bool first) {
            const uint32_t s = i & 1, par = (i >> 1) & 1;
            if (!wide_wait(sh, &sh.p_full[s], par) || !wide_wait(sh, &sh.v_full[s], par)) return false;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < BN / 16; ++q)
                mma_ts(tmem + S::kO, tmem + s * BN + 8 * q,
                       operand_desc(va + s * S::kStage + (q >> 2) * (D * 128) + (q & 3) * 32), wide_idesc(D),
                       !(first && q == 0));
            tc_commit(&sh.pv_done[s]);
            return true;
        };
        each_run([&](const Item<L> &, int, int k0, int k1, float *) {
            if (!wide_wait(sh, &sh.q_full, run & 1)) return false;
            ++run;
            for (int k = k0; k < k1; ++k, ++n) {
                const uint32_t s = n & 1, par = (n >> 1) & 1;
                // the weights of tile n - 2, which this S replaces, have been used up
                if (n >= 2 && !wide_wait(sh, &sh.pv_done[s], par ^ 1)) return false;
                if (!wide_wait(sh, &sh.k_full[s], par)) return false;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < D / 16; ++q)
                    mma_ss(tmem + s * BN, operand_desc(qa + (q >> 2) * (128 * 128) + (q & 3) * 32),
                           operand_desc(ka + s * S::kStage + (q >> 2) * (BN * 128) + (q & 3) * 32), wide_idesc(BN),
                           q != 0);
                tc_commit(&sh.s_full[s]);
                if (k > k0 && !value_product(n - 1, k - 1 == k0)) return false;
            }
            return value_product(n - 1, k1 - k0 == 1);
        });
        // nothing of this CTA is under way any more when its tensor memory goes back
        tc_commit(&sh.drained);
        mbar_wait_bounded(&sh.drained, 0, kWideTimeout, nullptr);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

int kv_attention_wide_status(unsigned int *out, int clear) {
    return kv_status_word(g_kv_attention_status, out, clear);
}

// ---- host --------------------------------------------------------------------------------------

template <int D, int BITS>
static int wide_launch_of(const KvAttnArgs &a, cudaStream_t st) {
    using S = WideShape<D, BITS>;
    static std::atomic<int> attr_done[kMaxDevices];
    const int dev = current_device_index();
    if (dev < 0 || dev >= kMaxDevices) return RN_ERR_DEVICE;
    const auto kernel = kv_attention_wide_kernel<D, BITS>;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess) {
            cudaGetLastError();
            return RN_ERR_DEVICE;
        }
        attr_done[dev].store(1, std::memory_order_release);
    }
    const int rc = launch_pdl(kernel, dim3(static_cast<unsigned>(a.grid)), dim3(kWideThreads), S::kSmem, st, a);
    if (rc != RN_OK) return rc;
    return join_launch<D, typename S::L>(a, st);
}

AttnPlan wide_plan(int sm_count, int64_t B, int group, int D, int64_t max_q_len) {
    AttnPlan p;
    p.q_tiles = (max_q_len * group + 127) / 128;
    p.grid = sm_count;
    p.prefix_bytes = ((B * p.q_tiles + 1) * 8 + 15) / 16 * 16;
    p.bytes = p.prefix_bytes + static_cast<int64_t>(p.grid) * 2 * 128 * (D + 2) * 4;
    return p;
}

int wide_launch(int D, int format, const KvAttnArgs &a, cudaStream_t st) {
    return kv_dispatch(D, format, [&](auto d, auto bits) { return wide_launch_of<d.value, bits.value>(a, st); });
}

}  // namespace rn
