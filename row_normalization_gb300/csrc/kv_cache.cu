// kv_cache.cu -- the quantised key/value cache: writing tokens of a packed QKV
// tensor into their slots, and reading ragged token ranges back as bf16
// (sm_103a).
//
// Both are single passes bound by HBM: a write reads 4 D bytes of keys and
// values a token and head and stores 2 (D * bits / 8 + D / 16); a read is the
// reverse.  Eight lanes own one token and head, key and value, and keep both in
// registers as chunks of eight consecutive dimensions (16 bytes of bf16, all of
// one scale group): D / 32 independent 16-byte accesses a lane, whole sectors on
// either side.  A key lane's codes are one run of the stored order as they are; a
// value lane's are after 4 x 4 transposes among its neighbours.
#include "kv_common.cuh"

namespace rn {

static __device__ unsigned int g_kv_cache_status = 0u;

constexpr int kKvThreads = 256;
constexpr int kRowLanes = 8;

// Lane l of a row's eight, chunk k: its first dimension, its group, and the lane
// masks over which the group's four chunks lie.
template <int D, bool VALUE>
struct RowLanes {
    static constexpr int kChunks = D / 64;
    static constexpr int kXor0 = 1, kXor1 = VALUE ? 4 : 2;
    __device__ static __forceinline__ int dim(int l, int k) {
        return VALUE ? 64 * k + 16 * (l & 3) + 8 * (l >> 2) : 32 * ((l >> 2) * kChunks + k) + 8 * (l & 3);
    }
};

// 4 x 4 transpose of the bytes (4 bits: a pair of codes each) or 16-bit units
// (8 bits) of a chunk among four lanes; its own inverse.
__device__ __forceinline__ void transpose4(uint32_t (&w)[1], int l) {
    // bytes: lane i's byte n <-> lane n's byte i, odd lanes first
    const uint32_t a = __shfl_xor_sync(0xffffffffu, w[0], 1);
    const uint32_t t = (l & 1) ? __byte_perm(a, w[0], 0x7351) : __byte_perm(w[0], a, 0x6240);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, t, 2);
    w[0] = (l & 2) ? __byte_perm(b, t, 0x7632) : __byte_perm(t, b, 0x5410);
}
__device__ __forceinline__ void transpose4(uint32_t (&w)[2], int l) {
    // units 0, 1 in w[0], 2, 3 in w[1]: halves of words with lane ^ 1, words with lane ^ 2
    const uint32_t a0 = __shfl_xor_sync(0xffffffffu, w[0], 1), a1 = __shfl_xor_sync(0xffffffffu, w[1], 1);
    const uint32_t t0 = (l & 1) ? __byte_perm(a0, w[0], 0x7632) : __byte_perm(w[0], a0, 0x5410);
    const uint32_t t1 = (l & 1) ? __byte_perm(a1, w[1], 0x7632) : __byte_perm(w[1], a1, 0x5410);
    const uint32_t b = __shfl_xor_sync(0xffffffffu, (l & 2) ? t0 : t1, 2);
    w[0] = (l & 2) ? b : t0;
    w[1] = (l & 2) ? t1 : b;
}

template <int WORDS>
__device__ __forceinline__ void store_words(uint32_t *dst, const uint32_t (&w)[WORDS]) {
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int k = 0; k < WORDS / 4; ++k)
            st16(dst + 4 * k, make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
    } else if constexpr (WORDS == 2) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    } else {
        static_assert(WORDS == 1, "one, two or a multiple of four words");
        dst[0] = w[0];
    }
}
template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&w)[WORDS], const uint32_t *src) {
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int k = 0; k < WORDS / 4; ++k) {
            const uint4 v = *reinterpret_cast<const uint4 *>(src + 4 * k);
            w[4 * k] = v.x;
            w[4 * k + 1] = v.y;
            w[4 * k + 2] = v.z;
            w[4 * k + 3] = v.w;
        }
    } else if constexpr (WORDS == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(src);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        static_assert(WORDS == 1, "one, two or a multiple of four words");
        w[0] = src[0];
    }
}

// ---- write ------------------------------------------------------------------------

// 1 / x to 2^-23, subnormal results as zero.
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Quantises a lane's chunks x and stores codes and scales of its row.
//   s = fp16(max|x| / Q), c = rne(x / s) clamped to +-Q.
// x * (1 / s) with a reciprocal good to 2^-22 is off by 2^-15 at most (|x / s| <
// 128 wherever the clamp does not decide).  x has 8 significant bits and s at most 11, so x / s is either
// exactly half way between two codes or at least 2^-12 away from there:
// rounding the product to a multiple of 2^-13 first (the fused multiply-add
// with 1536, whose last place that is) restores the exact tie, and the second
// rounding is then that of the true quotient.
template <int D, int BITS, bool VALUE>
__device__ __forceinline__ void quantise_row(const uint4 (&x)[D / 64], int l, const KvCache &cache, int64_t row,
                                             bool store) {
    using L = RowLanes<D, VALUE>;
    using F = KvFormat<D, BITS>;
    constexpr int CW = BITS / 4;  // words of a chunk's codes
    uint32_t out[L::kChunks * CW];
    uint16_t sb[L::kChunks];
#pragma unroll
    for (int k = 0; k < L::kChunks; ++k) {
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        // |x| as integers: the order of magnitudes, with infinities and NaNs on top
        uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, L::kXor0));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, L::kXor1));
        const uint32_t amax = max(top & 0xFFFFu, top >> 16);
        const bool finite = amax < 0x7F80u;
        const float a = __uint_as_float(amax << 16);
        // max|x| / Q is 2^-19 of itself away from every tie of fp16's normal numbers, so
        // the product's 2^-23 decides none; among the subnormal ones it can be a tie
        float d = a * (1.0f / F::kQ);
        if (a < F::kQ * 0x1.1p-14f) d = a / F::kQ;
        sb[k] = finite ? __half_as_ushort(__float2half_rn(fminf(d, 65504.0f))) : kKvNanScale;
        const float s = half_bits_to_float(sb[k]);
        const float inv = (finite && s > 0.0f) ? rcp_approx(s) : 0.0f;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            fma2(y[e], y[e + 1], bf_lo(w[e / 2]), bf_hi(w[e / 2]), inv, 1536.0f);
        // A normal fp16 scale is within 2^-11 of max|x| / Q, which leaves |x / s| under
        // Q + 0.07; only subnormal scales and the largest one need the clamp.
        if (sb[k] - 0x0400u > 0x7BFEu - 0x0400u) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fminf(fmaxf(y[e], 1536.0f - F::kQ), 1536.0f + F::kQ);
        }
        // adding 1.5 * 2^23 + zero - 1536 leaves the stored code in the low bits; the
        // codes are put together as sums, whose constant parts come off at the end
        uint32_t c[CW];
        constexpr uint32_t kMagic = 0x4B400000u;  // 1.5 * 2^23
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            uint32_t sum = 0u, extra = 0u;
#pragma unroll
            for (int e = 0; e < 32 / BITS; e += 2) {
                float z0, z1;
                const int n = i * (32 / BITS) + e;
                add2(z0, z1, y[n], y[n + 1], 12582912.0f + F::kZero - 1536.0f);
                sum += __float_as_uint(z0) << (e * BITS);
                sum += __float_as_uint(z1) << (e * BITS + BITS);
                extra += (kMagic << (e * BITS)) + (kMagic << (e * BITS + BITS));
            }
            constexpr uint32_t kNone = BITS == 4 ? 0x88888888u : 0x80808080u;  // all codes zero
            c[i] = finite ? sum - extra : kNone;
        }
        if constexpr (VALUE) transpose4(c, l);
#pragma unroll
        for (int i = 0; i < CW; ++i) out[k * CW + i] = c[i];
    }
    uint32_t *dst = reinterpret_cast<uint32_t *>(cache.codes + row * F::kRow);
    uint16_t *sdst = cache.scales + row * F::kGroups;
    if constexpr (VALUE) {
        // lane 0 holds the even groups' scales, lane 2 the odd ones'
        uint32_t sw[L::kChunks];
#pragma unroll
        for (int k = 0; k < L::kChunks; ++k) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, static_cast<uint32_t>(sb[k]), 2);
            sw[k] = sb[k] | other << 16;
        }
        if (store) {
            store_words(dst + l * (L::kChunks * CW), out);
            if (l == 0) store_words(reinterpret_cast<uint32_t *>(sdst), sw);
        }
    } else if (store) {
        // stored run: position l & 3 of four, groups (l >> 2) * kChunks ..
        store_words(dst + ((l & 3) * F::kGroups + (l >> 2) * L::kChunks) * CW, out);
        if ((l & 3) == 0) {
#pragma unroll
            for (int k = 0; k < L::kChunks; ++k) sdst[(l >> 2) * L::kChunks + k] = sb[k];
        }
    }
}

// A token's heads are taken kHeads at a time by one group of lanes, which shares
// the slot and the page among them.
template <int D, int BITS, int kHeads>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvWriteArgs a) {
    pdl_trigger();
    pdl_wait();
    const int l = static_cast<int>(threadIdx.x & (kRowLanes - 1));
    const uint32_t part = blockIdx.x * (kKvThreads / kRowLanes) + threadIdx.x / kRowLanes;
    const uint32_t t = part / a.parts;
    const int h0 = static_cast<int>(part - t * a.parts) * kHeads;
    int64_t slot = t < a.tokens ? a.slots[t] : -1;
    if (slot >= a.num_slots) {
        if (l == 0) atomicOr(&g_kv_cache_status, RN_STATUS_BAD_INDEX);
        slot = -1;
    }
    // a token without a slot: its lanes take part in the warp's shuffles only
    if (__all_sync(0xffffffffu, slot < 0)) return;
    const int64_t to_value = static_cast<int64_t>(a.cache.Hkv) * D;
    const uint16_t *src = a.kv + t * a.stride + static_cast<int64_t>(h0) * D;
    uint4 x[kHeads][2][D / 64];
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
            x[i][0][k] = x[i][1][k] = make_uint4(0u, 0u, 0u, 0u);
            if (slot >= 0 && h0 + i < a.cache.Hkv) {
                x[i][0][k] = ld_stream16(src + i * D + RowLanes<D, false>::dim(l, k));
                x[i][1][k] = ld_stream16(src + i * D + to_value + RowLanes<D, true>::dim(l, k));
            }
        }
    const int64_t row0 = slot >= 0 ? a.cache.row(slot >> a.cache.log2_page, 0, h0,
                                                 static_cast<int>(slot & ((1 << a.cache.log2_page) - 1)))
                                   : 0;
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const bool live = slot >= 0 && h0 + i < a.cache.Hkv;
        const int64_t row = row0 + (static_cast<int64_t>(i) << a.cache.log2_page);
        quantise_row<D, BITS, false>(x[i][0], l, a.cache, row, live);
        quantise_row<D, BITS, true>(x[i][1], l, a.cache,
                                    row + (static_cast<int64_t>(a.cache.Hkv) << a.cache.log2_page), live);
    }
}

// ---- read ---------------------------------------------------------------------

struct KvReadArgs {
    KvCache cache;
    const int32_t *page_table;  // [B, max_pages]
    int64_t B;
    int64_t max_pages;
    const int64_t *cu_lens;     // [B + 1]
    const int32_t *starts;      // [B] or null
    uint32_t rows;              // total
    uint32_t parts;             // groups of kHeads heads of a token
    uint16_t *out[2];           // k, v [total, Hkv, D]
};

// The last sequence whose first row is not behind row i (rows of empty
// sequences belong to nobody), or -1 for a row outside [cu[0], cu[B]).
__device__ __forceinline__ int64_t sequence_of_row(const int64_t *cu, int64_t B, int64_t i) {
    if (i < cu[0] || i >= cu[B]) return -1;
    int64_t lo = 0, hi = B - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Writes a lane's share of a row from its stored words and scales (dst null: a lane
// without a row, which only takes part in the shuffles).
template <int D, int BITS, bool VALUE>
__device__ __forceinline__ void restore_row(uint32_t (&c)[D / 64 * BITS / 4], const uint32_t (&sw)[D / 64], int l,
                                            uint16_t *dst) {
    using L = RowLanes<D, VALUE>;
    using F = KvFormat<D, BITS>;
    constexpr int CW = BITS / 4;
#pragma unroll
    for (int k = 0; k < L::kChunks; ++k) {
        uint32_t w[CW];
#pragma unroll
        for (int i = 0; i < CW; ++i) w[i] = c[k * CW + i];
        if constexpr (VALUE) transpose4(w, l);
        // group of the chunk: value 2k + (l & 3) / 2, key (l >> 2) * kChunks + k
        uint32_t pair;
        bool odd;
        if constexpr (VALUE) {
            pair = sw[k];
            odd = l & 2;
        } else if constexpr (L::kChunks == 1) {
            pair = sw[0];
            odd = l & 4;
        } else {
            pair = (l & 4) ? sw[(L::kChunks + k) / 2] : sw[k / 2];
            odd = k & 1;
        }
        const float s = half_bits_to_float(static_cast<uint16_t>(odd ? pair >> 16 : pair & 0xFFFFu));
        // codes to numbers: under the exponent of 1024 a code is 1024 + c in fp16, two
        // at a time, sixteen bits apart
        float x[8];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int i0 = BITS == 4 ? n : (n & 1) + 4 * (n >> 1), i1 = i0 + (BITS == 4 ? 4 : 2);
            const uint32_t m = BITS == 4 ? (w[0] >> (4 * n)) & 0x000F000Fu : (w[n >> (BITS / 8)] >> (8 * (n & 1))) & 0x00FF00FFu;
            const uint32_t u = m | 0x64006400u;
            const __half2 q = __hsub2(*reinterpret_cast<const __half2 *>(&u), __float2half2_rn(1024.0f + F::kZero));
            x[i0] = s * __low2float(q);
            x[i1] = s * __high2float(q);
        }
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = pack_bf2(x[2 * e], x[2 * e + 1]);
        if (dst) st16(dst + L::dim(l, k), make_uint4(y[0], y[1], y[2], y[3]));
    }
}

template <int D, int BITS, int kHeads>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvReadArgs a) {
    using F = KvFormat<D, BITS>;
    constexpr int CW = BITS / 4, CHUNKS = D / 64;
    pdl_trigger();
    pdl_wait();
    const int l = static_cast<int>(threadIdx.x & (kRowLanes - 1));
    const uint32_t part = blockIdx.x * (kKvThreads / kRowLanes) + threadIdx.x / kRowLanes;
    const uint32_t i = part / a.parts;
    const int h0 = static_cast<int>(part - i * a.parts) * kHeads;
    // offsets that name rows the results do not have
    if (part == 0 && l == 0 && (a.cu_lens[0] < 0 || a.cu_lens[a.B] > static_cast<int64_t>(a.rows)))
        atomicOr(&g_kv_cache_status, RN_STATUS_BAD_INDEX);
    const int64_t b = i < a.rows ? sequence_of_row(a.cu_lens, a.B, i) : -1;
    // lanes without a row take part in the warp's shuffles only
    if (__all_sync(0xffffffffu, b < 0)) return;
    int64_t token = 0, page = -1;
    if (b >= 0) {
        token = (a.starts ? a.starts[b] : 0) + (i - a.cu_lens[b]);
        const int64_t idx = token >> a.cache.log2_page;
        if (token >= 0 && idx < a.max_pages) page = a.page_table[b * a.max_pages + idx];
        if (page < 0 || page >= a.cache.num_pages) {
            page = -1;
            if (l == 0) atomicOr(&g_kv_cache_status, RN_STATUS_BAD_INDEX);
        }
    }
    uint32_t c[kHeads][2][CHUNKS * CW], sw[kHeads][2][F::kGroups / 2];
    const int64_t row0 =
        page >= 0 ? a.cache.row(page, 0, h0, static_cast<int>(token & ((1 << a.cache.log2_page) - 1))) : 0;
#pragma unroll
    for (int n = 0; n < kHeads; ++n)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
#pragma unroll
            for (int k = 0; k < CHUNKS * CW; ++k) c[n][which][k] = 0u;
#pragma unroll
            for (int k = 0; k < F::kGroups / 2; ++k) sw[n][which][k] = 0u;
            if (page >= 0 && h0 + n < a.cache.Hkv) {
                const int64_t r = row0 + (static_cast<int64_t>(n + which * a.cache.Hkv) << a.cache.log2_page);
                const int word = which ? l * (CHUNKS * CW) : ((l & 3) * F::kGroups + (l >> 2) * CHUNKS) * CW;
                load_words(c[n][which], reinterpret_cast<const uint32_t *>(a.cache.codes + r * F::kRow) + word);
                load_words(sw[n][which], reinterpret_cast<const uint32_t *>(a.cache.scales + r * F::kGroups));
            }
        }
    const int64_t out0 = (static_cast<int64_t>(i) * a.cache.Hkv + h0) * D;
#pragma unroll
    for (int n = 0; n < kHeads; ++n) {
        const bool live = b >= 0 && h0 + n < a.cache.Hkv;
        restore_row<D, BITS, false>(c[n][0], sw[n][0], l, live ? a.out[0] + out0 + n * D : nullptr);
        restore_row<D, BITS, true>(c[n][1], sw[n][1], l, live ? a.out[1] + out0 + n * D : nullptr);
    }
}

// ---- host ---------------------------------------------------------------------

// Heads that a group of lanes takes: two share the work of finding the row (16384
// tokens of 8 heads of 128, 4 bits: write 20.9 -> 17.6 us, read 16.0 -> 13.3), one
// where the registers of two cost more (256 wide: write 8.4 against 10.6 us), and one
// while all fit the GPU at once (64 tokens: write 2.4 against 3.2 us).
static int heads_at_once(const DeviceInfo &dev, int D, int64_t tokens, int Hkv) {
    const int64_t resident = static_cast<int64_t>(dev.sm_count) * 2048 / kRowLanes;
    return D == 256 || tokens * Hkv <= resident ? 1 : 2;
}
// Blocks of a launch over `parts` groups of heads of `rows` tokens each.
static dim3 row_grid(int64_t rows, int64_t parts) {
    constexpr int64_t per_block = kKvThreads / kRowLanes;
    return dim3(static_cast<unsigned>((rows * parts + per_block - 1) / per_block));
}

template <int D, int BITS, int HEADS>
static int write_launch(KvWriteArgs &a, cudaStream_t st) {
    a.parts = static_cast<uint32_t>((a.cache.Hkv + HEADS - 1) / HEADS);
    return launch_pdl(kv_write_kernel<D, BITS, HEADS>, row_grid(a.tokens, a.parts), dim3(kKvThreads), 0, st, a);
}
template <int D, int BITS, int HEADS>
static int read_launch(KvReadArgs &a, cudaStream_t st) {
    a.parts = static_cast<uint32_t>((a.cache.Hkv + HEADS - 1) / HEADS);
    return launch_pdl(kv_read_kernel<D, BITS, HEADS>, row_grid(a.rows, a.parts), dim3(kKvThreads), 0, st, a);
}

int kv_cache_status(unsigned int *out, int clear) {
    return kv_status_word(g_kv_cache_status, out, clear);
}

}  // namespace rn

extern "C" {

int kv_cache_write(const rn_bf16 *qkv, const int64_t *slots, int64_t T, int Hq, int Hkv, int D,
                   int format, int page_size, int64_t num_pages, uint8_t *codes, rn_f16 *scales,
                   rn_stream_t stream) {
    const int rc = rn::kv_check_sizes(format, Hkv, D, page_size, num_pages);
    if (rc != RN_OK) return rc;
    if (T < 0 || Hq < 0 || T > INT32_MAX / Hkv) return RN_ERR_SHAPE;
    if (T == 0) return RN_OK;
    if (!qkv || !slots || !codes || !scales) return RN_ERR_NULL;
    if (!rn::aligned16(qkv) || !rn::aligned16(codes) || !rn::aligned16(scales) ||
        (reinterpret_cast<uintptr_t>(slots) & 7u))
        return RN_ERR_ALIGN;
    const rn::DeviceInfo *dev = rn::current_device_info();
    if (!dev) return RN_ERR_DEVICE;
    rn::KvWriteArgs a;
    a.kv = qkv + static_cast<int64_t>(Hq) * D;
    a.stride = (static_cast<int64_t>(Hq) + 2 * static_cast<int64_t>(Hkv)) * D;
    a.slots = slots;
    a.tokens = static_cast<uint32_t>(T);
    a.cache = {codes, scales, num_pages, Hkv, rn::kv_log2_page(page_size)};
    a.num_slots = num_pages << a.cache.log2_page;
    const int heads = rn::heads_at_once(*dev, D, T, Hkv);
    const auto st = reinterpret_cast<cudaStream_t>(stream);
    return rn::kv_dispatch(D, format, [&](auto d, auto bits) {
        if constexpr (d.value != 256)
            if (heads == 2) return rn::write_launch<d.value, bits.value, 2>(a, st);
        return rn::write_launch<d.value, bits.value, 1>(a, st);
    });
}

int kv_cache_read(const uint8_t *codes, const rn_f16 *scales, int format, int Hkv, int D,
                  int page_size, int64_t num_pages, const int32_t *page_table, int64_t B,
                  int64_t max_pages, const int64_t *cu_lens, const int32_t *starts, int64_t total,
                  rn_bf16 *k, rn_bf16 *v, rn_stream_t stream) {
    const int rc = rn::kv_check_sizes(format, Hkv, D, page_size, num_pages);
    if (rc != RN_OK) return rc;
    if (B < 0 || B > INT32_MAX || max_pages < 0 || max_pages > INT32_MAX) return RN_ERR_SHAPE;
    if (total < 0 || total > INT32_MAX / Hkv) return RN_ERR_SHAPE;
    if (total == 0 || B == 0) return RN_OK;
    if (!codes || !scales || !cu_lens || !k || !v || (!page_table && max_pages > 0))
        return RN_ERR_NULL;
    if (!rn::aligned16(codes) || !rn::aligned16(scales) || !rn::aligned16(k) || !rn::aligned16(v) ||
        (reinterpret_cast<uintptr_t>(cu_lens) & 7u) ||
        ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(starts)) & 3u))
        return RN_ERR_ALIGN;
    if (k == v) return RN_ERR_ARG;
    const rn::DeviceInfo *dev = rn::current_device_info();
    if (!dev) return RN_ERR_DEVICE;
    rn::KvReadArgs a;
    a.cache = {const_cast<uint8_t *>(codes), const_cast<uint16_t *>(scales), num_pages, Hkv,
               rn::kv_log2_page(page_size)};
    a.page_table = page_table;
    a.B = B;
    a.max_pages = max_pages;
    a.cu_lens = cu_lens;
    a.starts = starts;
    a.rows = static_cast<uint32_t>(total);
    a.out[0] = k;
    a.out[1] = v;
    const int heads = rn::heads_at_once(*dev, D, total, Hkv);
    const auto st = reinterpret_cast<cudaStream_t>(stream);
    return rn::kv_dispatch(D, format, [&](auto d, auto bits) {
        if constexpr (d.value != 256)
            if (heads == 2) return rn::read_launch<d.value, bits.value, 2>(a, st);
        return rn::read_launch<d.value, bits.value, 1>(a, st);
    });
}

}  // extern "C"
