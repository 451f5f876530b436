// kv_attention.cu -- causal attention of ragged queries over the quantised
// key/value cache (sm_103a).
//
// The mathematics.  For a query q and visible tokens t with keys s_tg c_td
// (g = d / 32) and likewise values,
//   x_t = scale * sum_g s_tg sum_{d in g} q_d c_td,
//   out_d = sum_t 2^(y_t - r) s_tg c_td / sum_t 2^(y_t - r),  y = x log2(e).
// Both sums run on the tensor cores with the codes themselves as one operand:
// a code is an exact fp16 number, and so is the query (bf16, scaled by a power
// of two), so x_t has no rounding but that of fp32 sums.  The scales of the
// keys multiply fp32 partial sums of one group; the scales of the values
// multiply the weights before the second product.  Weight and product are fp16,
// which the tensor core takes at twice tf32's rate and half its registers: 2^-11
// relative each, within a range that attend_run keeps wide (64 sequences of 200 to 16000
// tokens, 4 bits: 4% of the time).
//
// Codes reach the tensor core without a conversion: a code c in the low bits
// of a 16-bit word is the subnormal fp16 number c * 2^-24, so masking a word
// of the stored row is all it takes (a 4-bit code four bits further up counts
// sixteen times; the query, or the finished sum, is divided by 16 there).
// The stored order puts the two halves of each operand register sixteen bits
// apart.  The offset of the stored codes (8 or 128) is taken off the sums
// where one instruction's operand serves few columns, else off the operands.
//
// What bounds it: a decode step reads every visible byte once (HBM).  The
// tokens are the rows of each product (16 an instruction) and the queries its
// columns (8, all heads of the group and all queries of the tile), so nothing
// is padded on the long side.
//
// Work is cut evenly over a fixed grid: all (sequence, query tile, kv head,
// 32-token tile) units form one line, of which every CTA takes an equal run,
// so ragged lengths leave no CTA behind.  Each (query tile, head) also has
// kLead units without work in front, for what it costs to begin and end one.  A
// run that cuts a (query tile, head) leaves partial sums in the workspace, which a
// second kernel joins in the order of the line.  Short contexts go without: a CTA
// for each (query tile, head), one launch (attn_direct).  Inside a CTA four warps
// take every fourth tile with an asynchronous copy ring of their own each and join at
// the end.  Calls that mix chunks with single tokens take two launches, each with the
// tile that fits its sequences (attn_mixed).
//
// Measured (one GB300, steady state): 64 sequences of 200 to 16000 tokens, 32 query and
// 8 kv heads of 128, 4 bits: 125 us, 5.0 TB/s of the bytes that have to be read; four of
// 131072 tokens 116 us, 5.2 TB/s; in 8 bits heads of 128 184 us, 6.4 TB/s, heads of 64
// (96 sequences) 98 us, 5.3 TB/s.  In 8 bits the bytes bound; in 4 bits the unpacking
// (about 640 instructions a warp and tile of 32 tokens, the integer pipe half full, 50 to
// 60% of the issue slots used by three warps a scheduler).
#include "kv_attention.cuh"

namespace rn {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr float kTop = 15.0f;        // weights stay below 2^kTop
constexpr float kSlack = 4.0f;       // powers of two a weight may grow before a rescale
// Units without work in front of each (query tile, head): its queries, first page and
// copies, and the joining of its warps.  64 ragged sequences of 8 heads (540k tokens):
// 145 us with none, 129 with 8, 124 with 16, 130 with 32; 4 long ones 116-118 throughout.
constexpr int kLead = 16 * 32;  // in tokens
constexpr int kMinTokens = 32 * kAttnWarps;  // a CTA's run is no shorter

// Shapes of an instantiation: NT * 8 columns (queries of the tile times heads).
template <int D, int BITS, int NT>
struct AttnShape {
    using F = KvFormat<D, BITS>;
    static constexpr int NQ = 8 * NT;
    // tokens a warp takes at once: 16 where 32 would leave room for one CTA an SM (heads of
    // 256 in 8 bits: 17 sequences, drafts of 3 to 5 tokens 51 against 61 us; 64 sequences,
    // one token each 63 against 66)
    static constexpr int kTile = D == 256 && BITS == 8 ? 16 : 32;
    using L = LineShape<NQ, kTile, kLead / kTile, kMinTokens / kTile>;
    static constexpr int MT = D / 16;                 // 16-row tiles of the value product
    static constexpr int kScaleRow = 2 * F::kGroups;  // bytes of a row's scales
    static constexpr int kCodesBytes = kTile * F::kRow;
    static constexpr int kScalesBytes = kTile * kScaleRow;
    static constexpr int kStage = 2 * (kCodesBytes + kScalesBytes);
    // the offset of the keys' codes comes off the sums, as their first addend (else off
    // the operands, which then serve several instructions)
    static constexpr bool kKeySums = NT == 1;
    // CTAs an SM is to hold: by registers (O alone is MT * NT * 4 a thread), fewer with
    // deeper rings in 8 bits, where the bytes bound (heads of 128, 64 sequences: 184 us
    // with two, 190 with three; heads of 64, 96 sequences: 90 with three, 91 with four; in
    // 4 bits 124 with three, 137 with two), and by shared memory for two stages
    static constexpr int kQuery = NQ * D * 2;  // the queries, as operand registers
    static constexpr int kRoom = 224 * 1024;
    static constexpr int stages_at(int ctas) { return ctas < 1 ? 0 : (kRoom / ctas - 2048 - kQuery) / (kAttnWarps * kStage); }
    static constexpr int kByRegs = MT * NT * 4 >= 64 ? 2 : (D == 64 ? 4 : 3) - (BITS == 8 ? 1 : 0);
    // 16-token halves of a tile taken at once: one where the registers hold no more (32
    // sequences, drafts of 3 to 8 tokens, heads of 128: in 4 bits 95 against 103 us, in 8
    // bits 104 against 149; one token a sequence 139 against 128)
    static constexpr int kStep = MT * NT >= 32 || D == 256 ? 1 : 2;
    static constexpr int kCtas = stages_at(kByRegs) >= 2         ? kByRegs
                                 : stages_at(kByRegs - 1) >= 2 ? kByRegs - 1
                                                               : kByRegs - 2;
    static constexpr int kStages = stages_at(kCtas) > 4 ? 4 : stages_at(kCtas);
    static_assert(kStages >= 2, "the ring needs two stages");
    static constexpr int kRing = kAttnWarps * kStages * kStage;
    static constexpr int kJoin = kAttnWarps * NQ * D * 4;  // the warps' sums, over the ring
    static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + kQuery;
    static constexpr int kSlot = NQ * (D + 2);  // floats of one partial result
};

// ---- instructions ---------------------------------------------------------------

// d = a b + c: a 16 x 16, b 16 x 8 (fp16), c and d 16 x 8 (fp32).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                        float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    mma_f16(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

// Transposes an 8 x 8 matrix of 16-bit elements held one row by four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t hsub2_bits(uint32_t a, uint32_t b) {
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 16 bytes global -> shared, of which `bytes` are read and the rest is zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int WORDS>
__device__ __forceinline__ void lds_words(uint32_t (&w)[WORDS], uint32_t addr) {
    if constexpr (WORDS == 1) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    } else if constexpr (WORDS == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    } else {
        static_assert(WORDS == 4, "one, two or four words");
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr));
    }
}

template <int WORDS>
__device__ __forceinline__ void sts_words(uint32_t addr, const uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 1) {
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(w[0]) : "memory");
    } else if constexpr (WORDS == 2) {
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(w[0]), "r"(w[1]) : "memory");
    } else {
        static_assert(WORDS == 4, "one, two or four words");
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3])
                     : "memory");
    }
}

// Byte offset of 16-byte chunk `chunk` of a tile's codes, token t at chunk
// t * ROW / 16.  The chunks of a 128-byte line are exchanged by a mask that
// depends on the line, so that both readers are free of bank conflicts: the
// key operand (8 tokens, 4 runs of a row each) and the value operand (4
// tokens, 8 runs each).  Masks found by trying all that are linear in the
// line's number.
// Sixteen tokens on, the mask is the same; 32 chunks on, it changes by a constant
// (swizzle_step), so both users keep one offset a lane.
template <int ROW>
struct Swizzle {
    static constexpr int m0 = ROW == 32 ? 4 : (ROW == 256 ? 1 : 2);
    static constexpr int m1 = ROW == 32 ? 0 : (ROW == 256 ? 1 : 4);
    static constexpr int m2 = ROW >= 128 ? (ROW == 256 ? 4 : 1) : 0;
    static constexpr int m3 = ROW == 256 ? 2 : 0;
};
template <int ROW>
__device__ __forceinline__ uint32_t swizzle(int chunk) {
    using W = Swizzle<ROW>;
    const int line = chunk >> 3;
    return 16 * (chunk ^ ((line & 1) * W::m0) ^ ((line >> 1 & 1) * W::m1) ^ ((line >> 2 & 1) * W::m2) ^
                 ((line >> 3 & 1) * W::m3));
}
// swizzle(32 i + lane) = 512 i + (swizzle(lane) ^ swizzle_step(i)), lane < 32.
template <int ROW>
constexpr uint32_t swizzle_step(int i) {
    return 16 * (((i & 1) * Swizzle<ROW>::m2) ^ ((i >> 1 & 1) * Swizzle<ROW>::m3));
}

// ---- the attention kernel ---------------------------------------------------------

// A column's query as operand registers and what goes with it.
template <int D, int BITS>
struct Query {
    using F = KvFormat<D, BITS>;
    uint32_t b[F::kGroups][2][2];  // [group][k-step][register]
    float sum[F::kGroups];         // of the lane's elements of a group
    float factor;                  // from a sum of codes * query to a logit in log2

    // Column `col` of the item, lane j of its four.  The query is scaled so that its
    // largest element lies in [2^13, 2^14): exact in fp16 down to 2^-28 of that.
    template <class L>
    __device__ __forceinline__ void load(const KvAttnArgs &a, const Item<L> &it, int head0, int col, int j) {
        uint32_t w[F::kGroups][4];
        uint32_t top = 0u;
        // (a query that sees no token counts as zeros, whatever it holds)
        const bool live = col < it.ncols && it.pos0 + (it.f0 + col) / a.group >= 0;
        const int f = it.f0 + (live ? col : 0);
        const uint16_t *src = a.q + (it.row0 + f / a.group) * a.q_stride +
                              static_cast<int64_t>(head0 + f % a.group) * D + 8 * j;
#pragma unroll
        for (int g = 0; g < F::kGroups; ++g) {
            const uint4 v = live ? ld_ro16(src + 32 * g) : make_uint4(0u, 0u, 0u, 0u);
            w[g][0] = v.x;
            w[g][1] = v.y;
            w[g][2] = v.z;
            w[g][3] = v.w;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[g][i] & 0x7FFF7FFFu);
        }
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t amax = max(top & 0xFFFFu, top >> 16);
        const bool finite = amax < 0x7F80u;
        int e = static_cast<int>(amax >> 7);   // biased exponent
        e = e < 14 ? 14 : e;
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(267 - (finite ? e : 127)) << 23),
                                   a.scale_log2);  // 2^(140 - e)
        // codes are c * 2^-24: factor = |scale| * 2^(e - 140 + 24)
        // (a negative scale turns the query's sign, and a zero one is as good as 2^-126:
        // the factor is positive, so it can multiply a maximum, or a masked -infinity)
        factor = fmaxf(ldexpf(fabsf(a.scale_log2), e - 116), 0x1p-126f);
        if (!finite) factor = __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int g = 0; g < F::kGroups; ++g) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = finite ? bf_lo(w[g][i]) * up : 0.0f;
                x[2 * i + 1] = finite ? bf_hi(w[g][i]) * up : 0.0f;
            }
            sum[g] = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
            if constexpr (BITS == 4) {
                b[g][0][0] = pack_h2(x[0], x[4]);
                b[g][0][1] = pack_h2(x[1] * 0.0625f, x[5] * 0.0625f);
                b[g][1][0] = pack_h2(x[2], x[6]);
                b[g][1][1] = pack_h2(x[3] * 0.0625f, x[7] * 0.0625f);
            } else {
                b[g][0][0] = pack_h2(x[0], x[2]);
                b[g][0][1] = pack_h2(x[1], x[3]);
                b[g][1][0] = pack_h2(x[4], x[6]);
                b[g][1][1] = pack_h2(x[5], x[7]);
            }
        }
    }
};

// Tiles [k0, k1) of one item and kv head: all warps, joined; the result goes to
// the output rows, or (part != null) unfinished into a slot of the workspace.
template <int D, int BITS, int NT>
__device__ __forceinline__ void attend_run(const KvAttnArgs &a,
                                           const Item<typename AttnShape<D, BITS, NT>::L> &it, int kvh,
                                           int k0, int k1, float *part, uint8_t *smem) {
    using S = AttnShape<D, BITS, NT>;
    using F = KvFormat<D, BITS>;
    constexpr int NG = F::kGroups;
    constexpr int NQ = S::NQ;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, j = lane & 3;
    __shared__ int s_pos[NQ];
    __shared__ float s_factor[NQ], s_ref[kAttnWarps][NQ], s_l[kAttnWarps][NQ];
    __shared__ float2 s_unit[kAttnWarps][S::kTile];  // of the tile's tokens: e, 2^-e

    // -- the warp's copy ring --------------------------------------------------------
    uint8_t *ring = smem + warp * (S::kStages * S::kStage);
    const uint32_t ring_addr = smem_addr(ring);
    const int log2_page = a.cache.log2_page;
    const int32_t *table = a.page_table + it.seq * a.max_pages;
    // the lane's first chunk in page 0 of this head, and the way to the next page and
    // from a key to its value
    constexpr int SCH = S::kScalesBytes / 16;  // chunks of a tile's key scales (then the values')
    const uint32_t copy_off = swizzle<F::kRow>(lane);
    // bytes of a page's codes and scales (keys, then values; under 4 GB by the host's check)
    const uint32_t page_codes = (static_cast<uint32_t>(2 * a.cache.Hkv) << log2_page) * F::kRow;
    const uint32_t page_scales = (static_cast<uint32_t>(2 * a.cache.Hkv) << log2_page) * S::kScaleRow;
    const int64_t head_row = static_cast<int64_t>(kvh) << log2_page;
    const uint8_t *codes0 = a.cache.codes + head_row * F::kRow + lane * 16;
    const uint8_t *scales0 = reinterpret_cast<const uint8_t *>(a.cache.scales) + head_row * S::kScaleRow +
                             (lane % SCH) * 16 + (SCH < 32 && lane >= SCH ? page_scales / 2 : 0);

    struct Pages {
        int lo, hi;  // of the tile's two halves (16 tokens each lie on one page)
    };
    const auto pages_of = [&](int k) {
        Pages p = {-1, -1};
        if (k < k1) {
            const int t0 = it.token(k);
            p.lo = table[t0 >> log2_page];
            if (S::kTile == 32 && log2_page == 4 && t0 + 16 < it.hi) p.hi = table[(t0 >> 4) + 1];
        }
        return p;
    };
    const auto seen = [&](int t) {  // some query sees a token of t .. t + 15
        return t < it.hi && (it.win_lo == 0 || t < a.sinks || t + 15 >= it.win_lo);
    };
    // Copies rows [FROM, TO) of a tile (halves or all of it), which lie on one page
    // starting at row `off` of it.  bytes = 0 writes zeros instead.
    const auto copy_rows = [&](auto from, auto to, uint32_t dst, uint32_t page, int off, int bytes) {
        constexpr int FROM = decltype(from)::value, TO = decltype(to)::value;
        constexpr int CPR = F::kRow / 16;  // chunks of a row, and copies a lane makes of a tile
        const uint8_t *src = codes0 + static_cast<uint64_t>(page) * page_codes + (off - FROM) * F::kRow;
        const uint8_t *vsrc = src + page_codes / 2;
#pragma unroll
        for (int i = CPR * FROM / 32; i < CPR * TO / 32; ++i) {
            const uint32_t d = dst + 512 * i + (copy_off ^ swizzle_step<F::kRow>(i));
            cp_async16(d, src + i * 512, bytes);
            cp_async16(d + S::kCodesBytes, vsrc + i * 512, bytes);
        }
        const uint8_t *ssrc = scales0 + static_cast<uint64_t>(page) * page_scales + (off - FROM) * S::kScaleRow;
        const uint32_t d = dst + 2 * S::kCodesBytes + lane * 16;
        if constexpr (SCH == 32) {
            if (FROM == 0 ? (TO == S::kTile || lane < 16) : lane >= 16) {
                cp_async16(d, ssrc, bytes);
                cp_async16(d + S::kScalesBytes, ssrc + page_scales / 2, bytes);
            }
        } else {
            const int c = lane % SCH;
            if (lane < 2 * SCH && (FROM == 0 ? (TO == S::kTile || c < SCH / 2) : c >= SCH / 2))
                cp_async16(d, ssrc, bytes);
        }
    };
    // Copies tile k into a stage.  Rows of a page that should be there and is not
    // arrive as zeros; what no query sees is masked, so whatever lies there will do.
    const auto issue = [&](int k, int stage, Pages p) {
        using I0 = std::integral_constant<int, 0>;
        using I16 = std::integral_constant<int, 16>;
        using I32 = std::integral_constant<int, 32>;
        const int t0 = it.token(k);
        const uint32_t dst = ring_addr + stage * S::kStage;
        const bool ok = static_cast<uint32_t>(p.lo) < static_cast<uint32_t>(a.cache.num_pages);
        if constexpr (S::kTile == 16) {
            if (!ok && lane == 0) atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
            copy_rows(I0(), I16(), dst, ok ? p.lo : 0, ok ? t0 & ((1 << log2_page) - 1) : 0, ok ? 16 : 0);
        } else if (log2_page > 4) {
            if (!ok && lane == 0) atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
            copy_rows(I0(), I32(), dst, ok ? p.lo : 0, ok ? t0 & ((1 << log2_page) - 1) : 0, ok ? 16 : 0);
        } else {
            const bool ok_hi = static_cast<uint32_t>(p.hi) < static_cast<uint32_t>(a.cache.num_pages);
            const bool see = seen(t0), see_hi = seen(t0 + 16);
            if (((see && !ok) || (see_hi && !ok_hi)) && lane == 0)
                atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
            if (see) copy_rows(I0(), I16(), dst, ok ? p.lo : 0, 0, ok ? 16 : 0);
            if (see_hi) copy_rows(I16(), I32(), dst, ok_hi ? p.hi : 0, 0, ok_hi ? 16 : 0);
        }
    };

    int k = k0 + warp;
    Pages next = pages_of(k);
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) {
        const int ks = k + s * kAttnWarps;
        if (ks < k1) issue(ks, s, next);
        next = pages_of(ks + kAttnWarps);
        cp_async_commit();
    }

    // -- queries ------------------------------------------------------------------
    const int head0 = kvh * a.group;
    float offset[S::kKeySums ? NG : 1][2];  // -zero * sum of the group's query, columns 2j, 2j+1
    float factor[NT][2];
    uint8_t *qsm = smem + (S::kSmem - S::kQuery);
    if (threadIdx.x < NQ)
        s_pos[threadIdx.x] = static_cast<int>(threadIdx.x) < it.ncols
                                 ? it.pos0 + (it.f0 + static_cast<int>(threadIdx.x)) / a.group
                                 : -1;
    if constexpr (S::kKeySums) {
        Query<D, BITS> q;
        q.load(a, it, head0, r, j);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float s = q.sum[g];
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            s *= -static_cast<float>(F::kZero) * 0x1p-24f;
            offset[g][0] = __shfl_sync(0xffffffffu, s, 8 * j);
            offset[g][1] = __shfl_sync(0xffffffffu, s, 8 * j + 4);
            if (warp == 0) {
                *reinterpret_cast<uint4 *>(qsm + (g * 32 + lane) * 16) =
                    make_uint4(q.b[g][0][0], q.b[g][0][1], q.b[g][1][0], q.b[g][1][1]);
            }
        }
        factor[0][0] = __shfl_sync(0xffffffffu, q.factor, 8 * j);
        factor[0][1] = __shfl_sync(0xffffffffu, q.factor, 8 * j + 4);
        __syncthreads();
    } else {
        for (int nt = warp; nt < NT; nt += kAttnWarps) {
            Query<D, BITS> q;
            q.load(a, it, head0, nt * 8 + r, j);
#pragma unroll
            for (int g = 0; g < NG; ++g)
                *reinterpret_cast<uint4 *>(qsm + ((nt * NG + g) * 32 + lane) * 16) =
                    make_uint4(q.b[g][0][0], q.b[g][0][1], q.b[g][1][0], q.b[g][1][1]);
            if (j == 0) s_factor[nt * 8 + r] = q.factor;
        }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            factor[nt][0] = s_factor[nt * 8 + 2 * j];
            factor[nt][1] = s_factor[nt * 8 + 2 * j + 1];
        }
    }

    // -- running state: column sums, and the finished product's rows ------------------
    float o[S::MT][NT][4], l[NT][2], m[NT][2], ref[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            l[nt][c] = 0.0f;
            m[nt][c] = -INFINITY;
            ref[nt][c] = 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < S::MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.0f;
    }
    // A token's weight counts 2^e and its values' scales 2^-e, with 2^e the power of two
    // above its largest scale in this head (2^-14 at least): scales lie below 1, and what
    // the weights are kept below, 2^kTop, bounds their products too.  m, ref and the fp16
    // weights are about weight * 2^e, so a token matters by what it adds to the result: one
    // of large weight and no value (a sink), or of huge values and no weight, takes no
    // bits from the others.
    // A new reference leaves the weights kSlack powers of two to grow, and is taken only when
    // that is used up: rescaling at every new maximum took 55% of the tiles of a ragged
    // decode batch.  So the largest is 2^11 at least, and 2^-25 of it is a normal number.

    // lane's places in a stage
    const int key_a = (r >> 1) + 4 * (r & 1);  // token of its first operand row
    constexpr int KW = NG * BITS / 4;          // words of a lane's share of a key row
    constexpr int VW = D * BITS / 256;         // and of a value row
    constexpr int KC = KW < 4 ? KW : 4, VC = VW < 4 ? VW : 4;
    // its chunk (and place in it) of token key_a and of that + 8; of tokens j + 4 n.
    // Further chunks of its share lie a constant away before the exchange: its share
    // starts at a multiple of its chunks, so they differ from the first in low bits only.
    uint32_t key_off[2], val_off[4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
        key_off[n] = swizzle<F::kRow>((key_a + 8 * n) * (F::kRow / 16) + j * KW / 4) + j * KW % 4 * 4;
#pragma unroll
    for (int n = 0; n < 4; ++n)
        val_off[n] = S::kCodesBytes + swizzle<F::kRow>((j + 4 * n) * (F::kRow / 16) + r * VW / 4) + r * VW % 4 * 4;

    // One tile: MASKED where some column does not see all of it.
    const auto do_tile = [&](auto masked_tag, uint32_t base, int t0) {
        constexpr bool MASKED = decltype(masked_tag)::value;
        const uint32_t sbase = base + 2 * S::kCodesBytes;
        // one token a lane: e and 2^-e for the warp, and its value scales times 2^-e in place
        if (S::kTile == 32 || lane < S::kTile) {
            constexpr int W = NG / 2;
            const uint32_t at = sbase + S::kScalesBytes + lane * S::kScaleRow;
            uint32_t v[W], mx = 0x04000400u;
            lds_words<W>(v, at);
            // (shifted by an exponent, so that infinity and NaN are negative integers)
#pragma unroll
            for (int i = 0; i < W; ++i) mx = __vmaxs2(mx, (v[i] & 0x7FFF7FFFu) + 0x04000400u);
            mx = __vmaxs2(mx, __byte_perm(mx, mx, 0x1032));
            const int e = static_cast<int>(mx >> 26) - 15;
            const float unit = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            const __half2 h = __float2half2_rn(unit);
#pragma unroll
            for (int i = 0; i < W; ++i) v[i] = hmul2_bits(v[i], *reinterpret_cast<const uint32_t *>(&h));
            sts_words<W>(at, v);
            s_unit[warp][lane] = make_float2(static_cast<float>(e), unit);
        }
        __syncwarp();
#pragma unroll 1
        for (int m0 = 0; m0 < S::kTile / 16; m0 += S::kStep) {
        // -- logits (before the factor): rows are tokens, columns queries --------------------------
        float x[S::kStep][NT][4];
#pragma unroll
        for (int mt = 0; mt < S::kStep; ++mt) {
            uint32_t ka[KW], kb[KW], sa[NG / 2], sb[NG / 2];
            const int ta = 16 * (m0 + mt) + key_a;
#pragma unroll
            for (int w = 0; w < KW; w += KC) {
                uint32_t v[KC];
                lds_words<KC>(v, base + 16 * (m0 + mt) * F::kRow + (key_off[0] ^ 4 * w));
#pragma unroll
                for (int i = 0; i < KC; ++i) ka[w + i] = v[i];
                lds_words<KC>(v, base + 16 * (m0 + mt) * F::kRow + (key_off[1] ^ 4 * w));
#pragma unroll
                for (int i = 0; i < KC; ++i) kb[w + i] = v[i];
            }
            lds_words<NG / 2>(sa, sbase + ta * S::kScaleRow);
            lds_words<NG / 2>(sb, sbase + (ta + 8) * S::kScaleRow);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[mt][nt][i] = 0.0f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                uint32_t f[2][4];  // operand registers of the group's two k-steps
                if constexpr (BITS == 4) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t wa = ka[g] >> (8 * s), wb = kb[g] >> (8 * s);
                        f[s][0] = wa & 0x000F000Fu;
                        f[s][1] = wb & 0x000F000Fu;
                        f[s][2] = wa & 0x00F000F0u;
                        f[s][3] = wb & 0x00F000F0u;
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        f[s][0] = ka[2 * g + s] & 0x00FF00FFu;
                        f[s][1] = kb[2 * g + s] & 0x00FF00FFu;
                        f[s][2] = (ka[2 * g + s] >> 8) & 0x00FF00FFu;
                        f[s][3] = (kb[2 * g + s] >> 8) & 0x00FF00FFu;
                    }
                }
                if constexpr (!S::kKeySums) {
                    constexpr uint32_t z = F::kZero * 0x00010001u, z2 = BITS == 4 ? 16 * z : z;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        f[s][0] = hsub2_bits(f[s][0], z);
                        f[s][1] = hsub2_bits(f[s][1], z);
                        f[s][2] = hsub2_bits(f[s][2], z2);
                        f[s][3] = hsub2_bits(f[s][3], z2);
                    }
                }
                const __half2 ha = *reinterpret_cast<const __half2 *>(&sa[g / 2]);
                const __half2 hb = *reinterpret_cast<const __half2 *>(&sb[g / 2]);
                const float fa = g & 1 ? __high2float(ha) : __low2float(ha);
                const float fb = g & 1 ? __high2float(hb) : __low2float(hb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 q = ld_shared16(qsm + ((nt * NG + g) * 32 + lane) * 16);
                    float d[4];
                    if constexpr (S::kKeySums)
                        mma_f16(d, f[0][0], f[0][1], f[0][2], f[0][3], q.x, q.y, offset[g][0], offset[g][1],
                                offset[g][0], offset[g][1]);
                    else
                        mma_f16(d, f[0][0], f[0][1], f[0][2], f[0][3], q.x, q.y, 0.0f, 0.0f, 0.0f, 0.0f);
                    mma_f16(d, f[1][0], f[1][1], f[1][2], f[1][3], q.z, q.w);
                    x[mt][nt][0] = fmaf(fa, d[0], x[mt][nt][0]);
                    x[mt][nt][1] = fmaf(fa, d[1], x[mt][nt][1]);
                    x[mt][nt][2] = fmaf(fb, d[2], x[mt][nt][2]);
                    x[mt][nt][3] = fmaf(fb, d[3], x[mt][nt][3]);
                }
            }
        }

        // -- mask ------------------------------------------------------------------------
        uint32_t hidden[NT];  // bit 4 mt + i: element x[mt][nt][i] is masked
        bool grow = false;
        if constexpr (MASKED) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                hidden[nt] = 0u;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int pos = s_pos[nt * 8 + 2 * j + c];
#pragma unroll
                    for (int mt = 0; mt < S::kStep; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int t = t0 + 16 * (m0 + mt) + 8 * h + key_a;
                            const bool see = t <= pos && (a.window == 0 || t > pos - a.window || t < a.sinks);
                            if (!see) {
                                x[mt][nt][2 * h + c] = -INFINITY;
                                hidden[nt] |= 1u << (4 * mt + 2 * h + c);
                            }
                        }
                }
            }
        }

        // -- running maximum, of the logits plus e ----------------------------------------
        float back[S::kStep][2];  // 2^-e of the lane's two tokens
#pragma unroll
        for (int mt = 0; mt < S::kStep; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 unit = s_unit[warp][16 * (m0 + mt) + 8 * h + key_a];
                back[mt][h] = unit.y;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        x[mt][nt][2 * h + c] = fmaf(x[mt][nt][2 * h + c], factor[nt][c], unit.x);
            }
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float t = fmaxf(x[0][nt][c], x[0][nt][2 + c]);
                if constexpr (S::kStep == 2) t = fmaxf(t, fmaxf(x[1][nt][c], x[1][nt][2 + c]));
                top[nt][c] = t;
                grow |= t > m[nt][c];  // m: the largest the reference allows
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float t = top[nt][c];
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    // columns that need no more room keep what they have
                    t = t > m[nt][c] ? t + kSlack : m[nt][c];
                    const float nref = t == -INFINITY ? 0.0f : t - kTop;
                    f[c] = m[nt][c] == -INFINITY ? 1.0f : exp2_approx(ref[nt][c] - nref);
                    ref[nt][c] = nref;
                    m[nt][c] = t;
                    l[nt][c] *= f[c];
                }
#pragma unroll
                for (int mt = 0; mt < S::MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][nt][i] *= f[i & 1];
            }
        }

        // -- weights: rounded once to fp16, then tokens along the operand's k --------------
        uint32_t p[S::kStep][NT][2];
#pragma unroll
        for (int mt = 0; mt < S::kStep; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = exp2_approx(x[mt][nt][i] - ref[nt][i & 1]);
                l[nt][0] = fmaf(w[0], back[mt][0], fmaf(w[2], back[mt][1], l[nt][0]));
                l[nt][1] = fmaf(w[1], back[mt][0], fmaf(w[3], back[mt][1], l[nt][1]));
                if constexpr (MASKED) {
                    // a masked weight is -0, so that it can be told from one that underflowed
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (hidden[nt] >> (4 * mt + i) & 1u) w[i] = -0.0f;
                }
                p[mt][nt][0] = transpose8(pack_h2(w[0], w[1]));
                p[mt][nt][1] = transpose8(pack_h2(w[2], w[3]));
            }

        // -- values: rows are dimensions, k tokens j, j + 4, j + 8, j + 12 -----------------
#pragma unroll
        for (int mt = 0; mt < S::kStep; ++mt) {
            uint32_t v[4][VW], vs[4][NG / 2];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int t = 16 * (m0 + mt) + 4 * n + j;
#pragma unroll
                for (int w = 0; w < VW; w += VC) {
                    uint32_t u[VC];
                    lds_words<VC>(u, base + 16 * (m0 + mt) * F::kRow + (val_off[n] ^ 4 * w));
#pragma unroll
                    for (int i = 0; i < VC; ++i) v[n][w + i] = u[i];
                }
                lds_words<NG / 2>(vs[n], sbase + S::kScalesBytes + t * S::kScaleRow);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t half = g & 1 ? 0x7632u : 0x5410u;
                const uint32_t s0 = __byte_perm(vs[0][g / 2], vs[1][g / 2], half);
                const uint32_t s1 = __byte_perm(vs[2][g / 2], vs[3][g / 2], half);
                uint32_t w0[NT], w1[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    w0[nt] = hmul2_bits(p[mt][nt][0], s0);
                    w1[nt] = hmul2_bits(p[mt][nt][1], s1);
                    if constexpr (MASKED) {  // a masked token's scale may be NaN
                        w0[nt] &= ~__vcmpeq2(p[mt][nt][0], 0x80008000u);
                        w1[nt] &= ~__vcmpeq2(p[mt][nt][1], 0x80008000u);
                    }
                }
#pragma unroll
                for (int hm = 0; hm < 2; ++hm) {
                    uint32_t f0, f1, f2, f3;
                    if constexpr (BITS == 4) {
                        const uint32_t c0 = __byte_perm(v[0][g / 2], v[1][g / 2], half) >> (8 * hm);
                        const uint32_t c1 = __byte_perm(v[2][g / 2], v[3][g / 2], half) >> (8 * hm);
                        f0 = c0 & 0x000F000Fu;
                        f1 = c0 & 0x00F000F0u;
                        f2 = c1 & 0x000F000Fu;
                        f3 = c1 & 0x00F000F0u;
                    } else {
                        const uint32_t c0 = __byte_perm(v[0][g], v[1][g], hm ? 0x7632u : 0x5410u);
                        const uint32_t c1 = __byte_perm(v[2][g], v[3][g], hm ? 0x7632u : 0x5410u);
                        f0 = c0 & 0x00FF00FFu;
                        f1 = (c0 >> 8) & 0x00FF00FFu;
                        f2 = c1 & 0x00FF00FFu;
                        f3 = (c1 >> 8) & 0x00FF00FFu;
                    }
                    constexpr uint32_t z = F::kZero * 0x00010001u, z2 = BITS == 4 ? 16 * z : z;
                    f0 = hsub2_bits(f0, z);
                    f1 = hsub2_bits(f1, z2);
                    f2 = hsub2_bits(f2, z);
                    f3 = hsub2_bits(f3, z2);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(o[2 * g + hm][nt], f0, f1, f2, f3, w0[nt], w1[nt]);
                }
            }
        }
        }
    };


    int stage = 0;
    for (; k < k1; k += kAttnWarps) {
        cp_async_wait<S::kStages - 2>();
        __syncwarp();
        {
            const int kn = k + (S::kStages - 1) * kAttnWarps;
            int sn = stage + S::kStages - 1;
            sn = sn >= S::kStages ? sn - S::kStages : sn;
            if (kn < k1) issue(kn, sn, next);
            next = pages_of(kn + kAttnWarps);
            cp_async_commit();
        }
        const uint32_t base = ring_addr + stage * S::kStage;
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
        const int t0 = it.token(k);

        const bool masked = t0 + S::kTile - 1 > it.lo_pos ||
                            (a.window && t0 <= it.hi - 1 - a.window && t0 + S::kTile > a.sinks);
        if (masked)
            do_tile(std::true_type(), base, t0);
        else
            do_tile(std::false_type(), base, t0);
    }

    // -- join the warps ---------------------------------------------------------------------
    cp_async_wait<0>();
    __syncthreads();  // every ring is idle: its space takes the sums
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float t = l[nt][c];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            const int col = nt * 8 + 2 * j + c;
            if (r == 0) {
                s_l[warp][col] = t;
                s_ref[warp][col] = m[nt][c] == -INFINITY ? -INFINITY : ref[nt][c];
            }
            if (col < it.ncols) {
#pragma unroll
                for (int mt = 0; mt < S::MT; ++mt) {
                    float e = o[mt][nt][c], d = o[mt][nt][2 + c];
                    if constexpr (BITS == 4) d *= 0.0625f;
                    *reinterpret_cast<float2 *>(sums + (warp * NQ + col) * D + 16 * mt + 2 * r) = make_float2(e, d);
                }
            }
        }
    __syncthreads();
    constexpr int QUADS = D / 4;  // threads of a column
    for (int idx = threadIdx.x; idx < it.ncols * QUADS; idx += kAttnThreads) {
        const int col = idx / QUADS, d0 = idx % QUADS * 4;
        float top = -INFINITY, l_all = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_ref[w][col]);
        const float base = top == -INFINITY ? 0.0f : top;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            const float f = exp2_approx(s_ref[w][col] - base);
            l_all = fmaf(s_l[w][col], f, l_all);
            const float4 v = *reinterpret_cast<const float4 *>(sums + (w * NQ + col) * D + d0);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        if (part) {
            *reinterpret_cast<float4 *>(part + col * D + d0) = acc;
            if (d0 == 0) {
                part[NQ * D + col] = top;
                part[NQ * D + NQ + col] = l_all;
            }
        } else {
            store_result<D>(a, it, head0, col, d0, acc, base, l_all);
        }
    }
    __syncthreads();  // the rings and the shared words are free again
}

template <int D, int BITS, int NT>
__global__ void __launch_bounds__(kAttnThreads, AttnShape<D, BITS, NT>::kCtas)
    kv_attention_kernel(const KvAttnArgs a) {
    using S = AttnShape<D, BITS, NT>;
    using L = typename S::L;
    extern __shared__ __align__(128) uint8_t attn_smem[];
    __shared__ int64_t scratch[kAttnWarps + 2];
    pdl_trigger();
    pdl_wait();
    int64_t item, before = 0, u = 0, u0 = 0, u1 = 1;
    Cut<L> cut(1, 1);
    if (a.direct) {
        item = blockIdx.x / static_cast<uint32_t>(a.cache.Hkv);
    } else {
        const Line line = find_unit<L, kAttnThreads>(a, blockIdx.x == 0, scratch);
        store_empty<D, L, kAttnThreads>(a);
        cut = Cut<L>(line.units, a.grid);
        if (line.units == 0 || blockIdx.x >= cut.ctas) return;
        u = u0 = cut.start(blockIdx.x);
        u1 = cut.start(blockIdx.x + 1);
        item = line.item;
        before = line.before;
    }
    while (u < u1) {
        const Item<L> it = make_item<L>(a, item);
        int head, k0, k1, v0 = 0, v1 = 1, units = 1;
        float *part = nullptr;
        if (a.direct) {
            head = static_cast<int>(blockIdx.x - static_cast<uint32_t>(item) * static_cast<uint32_t>(a.cache.Hkv));
            k0 = 0;
            k1 = it.n;
            if (it.bad && head == 0 && threadIdx.x == 0) atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
            if (it.n == 0) store_zeros<D, L, kAttnThreads>(a, it, head);
        } else {
            if (it.n == 0) {
                ++item;
                continue;
            }
            units = it.units();
            const int64_t in = u - before * a.cache.Hkv;
            head = static_cast<int>(quotient(in, units));
            v0 = static_cast<int>(in - static_cast<int64_t>(head) * units);
            const int64_t left = u1 - u;
            v1 = units - v0 <= left ? units : v0 + static_cast<int>(left);
            k0 = v0 > L::LEAD ? v0 - L::LEAD : 0;
            k1 = v1 - L::LEAD;
            if (k1 - k0 != it.n)
                part = a.partial + (2 * static_cast<int64_t>(blockIdx.x) + (u == u0 ? 0 : 1)) * S::kSlot;
        }
        if (k1 > k0) attend_run<D, BITS, NT>(a, it, head, k0, k1, part, attn_smem);
        if (!a.direct && threadIdx.x == 0) note_piece(a, cut, blockIdx.x, u - v0, v0, v1, units, it, item, head);
        u += v1 - v0;
        if (v1 == units && head == a.cache.Hkv - 1) {
            before += units;
            ++item;
        }
    }
}

int kv_attention_status(unsigned int *out, int clear) {
    return kv_status_word(g_kv_attention_status, out, clear);
}

// ---- host -------------------------------------------------------------------------------

// More columns than this go to the kernel that takes 128 of them at a time (16 sequences
// of 3000 to 8000 tokens, 8 heads; this kernel against that one, us: heads of 128 in 4
// bits, 64 columns 132 / 157, 128 columns 243 / 166; heads of 64 in 8 bits 76 / 107 and
// 139 / 111; heads of 256 in 4 bits 256 / 324 and 493 / 337).
static bool wide(int64_t columns) { return columns > 64; }

// Columns of a query tile, in eights: the smallest that holds all queries of a
// sequence times the heads of a group, else the largest the registers hold.
static int attn_tiles(int D, int64_t columns) {
    if (columns <= 8) return 1;
    if (columns <= 16 || D == 256) return 2;
    return 4;
}

template <int D, int BITS, int NT>
static AttnPlan attn_plan_of(int sm_count, int64_t B, int group, int64_t max_q_len) {
    using S = AttnShape<D, BITS, NT>;
    AttnPlan p;
    p.q_tiles = (max_q_len * group + S::NQ - 1) / S::NQ;
    p.grid = sm_count * S::kCtas;
    p.head_bytes = 16 + 32 * static_cast<int64_t>(p.grid);
    p.bytes = p.head_bytes + static_cast<int64_t>(p.grid) * 2 * S::kSlot * 4;
    return p;
}

// Calls f with the compile-time D, BITS and NT of a checked call.
template <typename Fn>
static auto attn_dispatch(int D, int format, int64_t columns, Fn &&f) {
    const int nt = attn_tiles(D, columns);
    return kv_dispatch(D, format, [&](auto d, auto bits) {
        if (nt == 1) return f(d, bits, std::integral_constant<int, 1>());
        if (nt == 2) return f(d, bits, std::integral_constant<int, 2>());
        if constexpr (d.value == 256) {
            return f(d, bits, std::integral_constant<int, 2>());
        } else {
            return f(d, bits, std::integral_constant<int, 4>());
        }
    });
}

// The plan of one launch for sequences of up to max_q_len queries.
static AttnPlan attn_plan(int sm_count, int format, int64_t B, int group, int D, int64_t max_q_len) {
    if (wide(max_q_len * group)) return wide_plan(sm_count, B, group, D, max_q_len);
    return attn_dispatch(D, format, max_q_len * group, [&](auto d, auto bits, auto nt) {
        return attn_plan_of<d.value, bits.value, nt.value>(sm_count, B, group, max_q_len);
    });
}

// Up to how many queries a sequence may go to a launch of its own: eight columns, or one
// token; 0 where max_q_len's kernel is the same, or takes 16 columns (single tokens pay
// for that: 64 of them over 4000 to 16000 tokens, 4 bits, 211 us where max_q_len is 4, 152
// where it is 1).
static int64_t attn_few(int D, int group, int64_t max_q_len) {
    const int64_t few = group < 8 ? 8 / group : 1, columns = few * group, most = max_q_len * group;
    if (wide(columns) || max_q_len <= few) return 0;
    return wide(most) || (attn_tiles(D, most) == 4 && attn_tiles(D, columns) != 4) ? few : 0;
}

// Whether each (query tile, head) gets a CTA of its own: no line, no joining.  Where no
// CTA can meet more than 1024 tokens, or 2048 and there are heads to fill the GPU (one
// token a sequence, 4 bits, 8 heads of 128, us on the line / directly: 4 sequences of up
// to 700 tokens 10.3 / 7.8, 256 of up to 900 55 / 50; of 300 to 1900 tokens 16
// sequences 15.8 / 18.2, 64 of them 30.6 / 30.4; of 1000 to 4000, 16: 25 / 36).
static bool attn_direct(const KvAttnArgs &a, int columns) {
    const int64_t most = attn_most_tokens(a, columns), busy = attn_busy_heads(a, columns);
    if (a.heads > 2 * busy || a.heads > INT32_MAX) return false;  // a grid of CTAs without work
    return most <= 1024 || (most <= 2048 && 3 * busy >= 2 * static_cast<int64_t>(a.grid));
}

template <int D, int BITS, int NT>
static int attn_launch(KvAttnArgs &a, cudaStream_t st) {
    using S = AttnShape<D, BITS, NT>;
    a.direct = attn_direct(a, S::NQ);
    static std::atomic<int> attr_done[kMaxDevices];
    const int dev = current_device_index();
    if (dev < 0 || dev >= kMaxDevices) return RN_ERR_DEVICE;
    const auto kernel = kv_attention_kernel<D, BITS, NT>;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess) {
            cudaGetLastError();
            return RN_ERR_DEVICE;
        }
        attr_done[dev].store(1, std::memory_order_release);
    }
    const unsigned ctas = static_cast<unsigned>(a.direct ? a.heads : a.grid);
    const int rc = launch_pdl(kernel, dim3(ctas), dim3(kAttnThreads), S::kSmem, st, a);
    if (rc != RN_OK || a.direct) return rc;
    return join_launch<D, typename S::L>(a, st);
}

// Workspace of a call, whichever launches it takes; one for max_q_len queries also serves
// calls of fewer, whose kernels may have more CTAs: the most of all up to as many columns.
static int64_t attn_bytes(int sm_count, int format, int64_t B, int group, int D, int64_t max_q_len) {
    const int64_t columns = max_q_len * group;
    int64_t most = 0;
    for (const int64_t c : {static_cast<int64_t>(8), static_cast<int64_t>(16), static_cast<int64_t>(64),
                            static_cast<int64_t>(128), columns}) {
        const int64_t bytes = attn_plan(sm_count, format, B, 1, D, c < columns ? c : columns).bytes;
        most = bytes > most ? bytes : most;
    }
    return most;
}

// Whether sequences of few queries get a launch of their own, before the others': where
// there are at most half as many queries as max_q_len allows (some sequences then have
// far fewer than others), and sequences enough to pay for the second launch.  One chunk
// of n queries among sequences of one (32 and 8 heads of 128 in 4 bits, contexts of up
// to 2000 tokens, us in one / in two): 64 sequences, n 12 85 / 69, 60 185 / 94, 500 294 /
// 109; 16, n 12 33 / 44, 60 77 / 64, 500 121 / 82; 4, n 60 39 / 51, 500 78 / 76.
static bool attn_mixed(const KvAttnArgs &a, int64_t few, int sm_count) {
    if (few == 0 || !a.cu_q || 2 * a.T > a.B * a.max_q_len) return false;
    const int64_t heads = (a.T < a.B ? a.T : a.B) * a.cache.Hkv;  // that may have a query
    return wide(a.max_q_len * a.group) ? 4 * heads >= 3 * static_cast<int64_t>(sm_count)
                                       : heads >= 2 * static_cast<int64_t>(sm_count);
}

// The launches for the sequences of min_q to most_q queries.
static int attn_pass(KvAttnArgs a, int sm_count, int D, int format, int64_t min_q, int64_t most_q, int64_t max_q_len,
                     void *workspace, cudaStream_t st) {
    const AttnPlan plan = attn_plan(sm_count, format, a.B, a.group, D, max_q_len);
    a.min_q = min_q;
    a.most_q = most_q;
    a.max_q_len = max_q_len;
    a.units = static_cast<int64_t *>(workspace);
    a.cuts = reinterpret_cast<CutNote *>(static_cast<char *>(workspace) + 16);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan.head_bytes);
    a.q_tiles = plan.q_tiles;
    a.heads = a.B * plan.q_tiles * a.cache.Hkv;
    a.grid = plan.grid;
    if (wide(max_q_len * a.group)) return wide_launch(D, format, a, st);
    return attn_dispatch(D, format, max_q_len * a.group, [&](auto d, auto bits, auto nt) {
        return attn_launch<d.value, bits.value, nt.value>(a, st);
    });
}

static int kv_attention_check(int format, int64_t B, int Hq, int Hkv, int D, int64_t max_q_len) {
    const int rc = kv_check_sizes(format, Hkv, D, 16, 1);
    if (rc != RN_OK) return rc;
    if (Hq < 1 || Hq > 65535 || Hq % Hkv != 0) return RN_ERR_SHAPE;
    if (B < 0 || B > INT32_MAX / Hq || max_q_len < 0 || max_q_len > INT32_MAX / Hq) return RN_ERR_SHAPE;
    // make_item counts (sequence, query tile)s in 31 bits, tiles of eight columns at least
    if (B > 0 && (max_q_len * (Hq / Hkv) + 7) / 8 > INT32_MAX / B) return RN_ERR_SHAPE;
    return RN_OK;
}

}  // namespace rn

extern "C" {

int64_t kv_attention_workspace_bytes(int format, int64_t B, int Hq, int Hkv, int D,
                                     int64_t max_q_len) {
    const int rc = rn::kv_attention_check(format, B, Hq, Hkv, D, max_q_len);
    if (rc != RN_OK) return rc;
    const rn::DeviceInfo *dev = rn::current_device_info();
    if (!dev) return RN_ERR_DEVICE;
    if (B == 0 || max_q_len == 0) return 16;
    return rn::attn_bytes(dev->sm_count, format, B, Hq / Hkv, D, max_q_len);
}

int kv_attention_fwd(const rn_bf16 *q, int64_t q_stride, const uint8_t *codes,
                     const rn_f16 *scales, int format, int Hq, int Hkv, int D, int page_size,
                     int64_t num_pages, const int32_t *page_table, int64_t B, int64_t max_pages,
                     const int32_t *kv_lens, const int64_t *cu_q, int64_t T, int64_t max_q_len,
                     float scale, int64_t window, int64_t sinks, rn_bf16 *out, float *lse,
                     void *workspace, int64_t workspace_bytes, rn_stream_t stream) {
    int rc = rn::kv_check_sizes(format, Hkv, D, page_size, num_pages);
    if (rc != RN_OK) return rc;
    rc = rn::kv_attention_check(format, B, Hq, Hkv, D, max_q_len);
    if (rc != RN_OK) return rc;
    const int log2_page = rn::kv_log2_page(page_size);
    if (T < 0 || T > INT32_MAX / Hq || max_pages < 0 || max_pages > (INT32_MAX >> log2_page))
        return RN_ERR_SHAPE;
    if (window < 0 || sinks < 0 || !(scale - scale == 0.0f)) return RN_ERR_ARG;
    if (!cu_q && T != B) return RN_ERR_SHAPE;
    if (q_stride < static_cast<int64_t>(Hq) * D || q_stride % 8 != 0) return RN_ERR_SHAPE;
    if (T == 0 || B == 0 || max_q_len == 0) return RN_OK;
    if (!q || !codes || !scales || !kv_lens || !out || !workspace || (!page_table && max_pages > 0))
        return RN_ERR_NULL;
    if (!rn::aligned16(q) || !rn::aligned16(codes) || !rn::aligned16(scales) ||
        !rn::aligned16(out) || !rn::aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(cu_q) & 7u) ||
        ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(kv_lens) |
          reinterpret_cast<uintptr_t>(lse)) & 3u))
        return RN_ERR_ALIGN;
    const rn::DeviceInfo *dev = rn::current_device_info();
    if (!dev) return RN_ERR_DEVICE;
    if (workspace_bytes < rn::attn_bytes(dev->sm_count, format, B, Hq / Hkv, D, max_q_len)) return RN_ERR_ARG;
    rn::KvAttnArgs a;
    a.q = q;
    a.q_stride = q_stride;
    a.cache = {const_cast<uint8_t *>(codes), const_cast<uint16_t *>(scales), num_pages, Hkv,
               log2_page};
    a.page_table = page_table;
    a.B = B;
    a.max_pages = max_pages;
    a.kv_lens = kv_lens;
    a.cu_q = cu_q;
    a.T = T;
    a.max_q_len = max_q_len;
    a.Hq = Hq;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.group = Hq / Hkv;
    a.window = static_cast<int>(window < INT32_MAX ? window : INT32_MAX);
    a.sinks = static_cast<int>(sinks < INT32_MAX ? sinks : INT32_MAX);
    a.out = out;
    a.lse = lse;
    const auto st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t few = rn::attn_few(D, a.group, max_q_len);
    if (!rn::attn_mixed(a, few, dev->sm_count))
        return rn::attn_pass(a, dev->sm_count, D, format, 0, INT64_MAX, max_q_len, workspace, st);
    rc = rn::attn_pass(a, dev->sm_count, D, format, 0, few, few, workspace, st);
    if (rc != RN_OK) return rc;
    return rn::attn_pass(a, dev->sm_count, D, format, few + 1, INT64_MAX, max_q_len, workspace, st);
}

}  // extern "C"
