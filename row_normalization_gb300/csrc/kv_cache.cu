// kv_cache.cu -- the quantised key/value cache: writing tokens of a packed QKV
// tensor into their slots, and reading ragged token ranges back as bf16
// (sm_103a).
//
// Both are single passes bound by HBM: a write reads 4 D bytes of keys and
// values a token and head and stores 2 (D * bits / 8 + D / 16); a read is the
// reverse.  A row (one token's key or value head) belongs to a group of lanes
// that keeps it in registers: 4 lanes for a key row and 8 for a value row, so
// that each lane's codes are one run of bytes of the stored order.
#include "kv_common.cuh"

namespace rn {

static __device__ unsigned int g_kv_cache_status = 0u;

constexpr int kKvThreads = 256;

// Lanes of a row and the dimensions of a lane's run k of consecutive elements:
//   key rows:   lane j of 4 holds, of every group g, dimensions 32g + 8j .. +7;
//   value rows: lane r of 8 holds, of every 16 dimensions b, 16b + 2r .. +1.
// E elements a lane, in RUNS runs of LEN; a run lies inside one scale group.
template <int D, bool VALUE>
struct RowLanes {
    static constexpr int kLanes = VALUE ? 8 : 4;
    static constexpr int E = D / kLanes;
    static constexpr int LEN = VALUE ? 2 : 8;
    static constexpr int RUNS = E / LEN;
    static constexpr int kRunsPerGroup = VALUE ? 2 : 1;
    __device__ static __forceinline__ int dim(int lane, int run) {
        return VALUE ? 16 * run + 2 * lane : 32 * run + 8 * lane;
    }
};

struct KvWriteArgs {
    const uint16_t *kv;    // first key element of token 0
    int64_t stride;        // elements from one token to the next
    const int64_t *slots;
    int64_t T;
    int64_t num_slots;
    KvCache cache;
};

// Quantises one row held as raw bf16 words w[E / 2] by kLanes lanes and stores it.
//   s = fp16(max|x| / Q), c = rne(x / s) clamped to +-Q.
// x * (1 / s) is off by 2^-17 at most (|x / s| < 128 wherever the clamp does
// not decide).  x has 8 significant bits and s at most 11, so x / s is either
// exactly half way between two codes or at least 2^-12 away from there:
// rounding the product to a multiple of 2^-13 first (the fused multiply-add
// with 1536, whose last place that is) restores the exact tie, and the second
// rounding is then that of the true quotient.
template <int D, int BITS, bool VALUE>
__device__ __forceinline__ void quantise_row(const uint32_t (&w)[RowLanes<D, VALUE>::E / 2],
                                             int lane, uint8_t *codes, uint16_t *scales,
                                             bool store) {
    using L = RowLanes<D, VALUE>;
    using F = KvFormat<D, BITS>;
    constexpr int PER_GROUP = kKvGroup / L::kLanes;  // elements a lane holds of a group
    uint32_t out[L::E * BITS / 32];
#pragma unroll
    for (int k = 0; k < L::E * BITS / 32; ++k) out[k] = 0u;
#pragma unroll
    for (int g = 0; g < F::kGroups; ++g) {
        // |x| as integers: the order of magnitudes, with infinities and NaNs on top
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < PER_GROUP / 2; ++i)
            top = __vmaxu2(top, w[g * (PER_GROUP / 2) + i] & 0x7FFF7FFFu);
#pragma unroll
        for (int o = L::kLanes / 2; o > 0; o >>= 1)
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        const uint32_t amax = max(top & 0xFFFFu, top >> 16);
        const bool finite = amax < 0x7F80u;
        const float a = __uint_as_float(amax << 16);
        const uint16_t sb = finite ? __half_as_ushort(__float2half_rn(
                                         fminf(a / static_cast<float>(F::kQ), 65504.0f)))
                                   : kKvNanScale;
        const float s = half_bits_to_float(sb);
        const float inv = (finite && s > 0.0f) ? 1.0f / s : 0.0f;
        if (lane == 0 && store) scales[g] = sb;
#pragma unroll
        for (int i = 0; i < PER_GROUP; ++i) {
            const int e = g * PER_GROUP + i;
            const float x = (e & 1) ? bf_hi(w[e / 2]) : bf_lo(w[e / 2]);
            float q = __fmaf_rn(x, inv, 1536.0f) - 1536.0f;
            q = fminf(fmaxf(q, -static_cast<float>(F::kQ)), static_cast<float>(F::kQ));
            q = finite ? q : 0.0f;
            // 1.5 * 2^23 plus the zero code: the sum's low bits are the stored code
            const uint32_t c = __float_as_uint(q + (12582912.0f + F::kZero)) & ((1u << BITS) - 1u);
            out[e * BITS / 32] |= c << (e * BITS % 32);
        }
    }
    constexpr int WORDS = L::E * BITS / 32;
    if (!store) return;
    uint32_t *dst = reinterpret_cast<uint32_t *>(codes) + lane * WORDS;
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int k = 0; k < WORDS / 4; ++k)
            st16(dst + 4 * k, make_uint4(out[4 * k], out[4 * k + 1], out[4 * k + 2], out[4 * k + 3]));
    } else if constexpr (WORDS == 2) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0], out[1]);
    } else {
        static_assert(WORDS == 1, "a lane's codes fill one, two or a multiple of four words");
        dst[0] = out[0];
    }
}

// blockIdx.y 0 writes the key rows, 1 the value rows.  256 threads take 64 key
// rows or 32 value rows: consecutive rows are the heads of one token, whose
// loads are therefore one contiguous run.
template <int D, int BITS, bool VALUE>
__device__ __forceinline__ void write_rows(const KvWriteArgs &a) {
    using L = RowLanes<D, VALUE>;
    using F = KvFormat<D, BITS>;
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kKvThreads + threadIdx.x;
    const int lane = static_cast<int>(gid) & (L::kLanes - 1);
    const int64_t row = gid / L::kLanes;
    const int64_t t = row / a.cache.Hkv;
    const int h = static_cast<int>(row - t * a.cache.Hkv);
    int64_t slot = t < a.T ? a.slots[t] : -1;
    if (slot >= a.num_slots) {
        if (lane == 0) atomicOr(&g_kv_cache_status, RN_STATUS_BAD_INDEX);
        slot = -1;
    }
    // a row without a slot: its lanes take part in the warp's shuffles only
    if (__all_sync(0xffffffffu, slot < 0)) return;
    const bool live = slot >= 0;
    uint32_t w[L::E / 2];
    const uint16_t *src =
        a.kv + t * a.stride + (static_cast<int64_t>(VALUE ? a.cache.Hkv : 0) + h) * D;
#pragma unroll
    for (int k = 0; k < L::RUNS; ++k) {
        if constexpr (VALUE) {
            w[k] = live ? *reinterpret_cast<const uint32_t *>(src + L::dim(lane, k)) : 0u;
        } else {
            const uint4 v = live ? ld_stream16(src + L::dim(lane, k)) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * k] = v.x;
            w[4 * k + 1] = v.y;
            w[4 * k + 2] = v.z;
            w[4 * k + 3] = v.w;
        }
    }
    const int64_t r = live ? a.cache.row(slot >> a.cache.log2_page, VALUE, h,
                                         static_cast<int>(slot & ((1 << a.cache.log2_page) - 1)))
                           : 0;
    quantise_row<D, BITS, VALUE>(w, lane, a.cache.codes + r * F::kRow,
                                 a.cache.scales + r * F::kGroups, live);
}

template <int D, int BITS>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(KvWriteArgs a) {
    pdl_trigger();
    pdl_wait();
    if (blockIdx.y == 0)
        write_rows<D, BITS, false>(a);
    else
        write_rows<D, BITS, true>(a);
}

// ---- read ---------------------------------------------------------------------

struct KvReadArgs {
    KvCache cache;
    const int32_t *page_table;  // [B, max_pages]
    int64_t B;
    int64_t max_pages;
    const int64_t *cu_lens;     // [B + 1]
    const int32_t *starts;      // [B] or null
    int64_t total;
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

template <int D, int BITS, bool VALUE>
__device__ __forceinline__ void read_rows(const KvReadArgs &a) {
    using L = RowLanes<D, VALUE>;
    using F = KvFormat<D, BITS>;
    constexpr int WORDS = L::E * BITS / 32;
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kKvThreads + threadIdx.x;
    const int lane = static_cast<int>(gid) & (L::kLanes - 1);
    const int64_t row = gid / L::kLanes;
    const int64_t i = row / a.cache.Hkv;
    const int h = static_cast<int>(row - i * a.cache.Hkv);
    if (i >= a.total) return;
    const int64_t b = sequence_of_row(a.cu_lens, a.B, i);
    if (b < 0) return;
    const int64_t token = (a.starts ? a.starts[b] : 0) + (i - a.cu_lens[b]);
    const int64_t idx = token >> a.cache.log2_page;
    int64_t page = -1;
    if (token >= 0 && idx < a.max_pages) page = a.page_table[b * a.max_pages + idx];
    uint32_t c[WORDS];
    uint16_t sb[F::kGroups];
    if (page >= 0 && page < a.cache.num_pages) {
        const int64_t r = a.cache.row(page, VALUE, h,
                                      static_cast<int>(token & ((1 << a.cache.log2_page) - 1)));
        const uint32_t *src =
            reinterpret_cast<const uint32_t *>(a.cache.codes + r * F::kRow) + lane * WORDS;
        const uint16_t *sc = a.cache.scales + r * F::kGroups;
        if constexpr (WORDS % 4 == 0) {
#pragma unroll
            for (int k = 0; k < WORDS / 4; ++k) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src + 4 * k);
                c[4 * k] = v.x;
                c[4 * k + 1] = v.y;
                c[4 * k + 2] = v.z;
                c[4 * k + 3] = v.w;
            }
        } else if constexpr (WORDS == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(src);
            c[0] = v.x;
            c[1] = v.y;
        } else {
            c[0] = src[0];
        }
#pragma unroll
        for (int g = 0; g < F::kGroups; ++g) sb[g] = sc[g];
    } else {
        if (lane == 0) atomicOr(&g_kv_cache_status, RN_STATUS_BAD_INDEX);
#pragma unroll
        for (int k = 0; k < WORDS; ++k) c[k] = 0u;
#pragma unroll
        for (int g = 0; g < F::kGroups; ++g) sb[g] = 0;
    }
    uint16_t *dst = a.out[VALUE] + row * D;
#pragma unroll
    for (int k = 0; k < L::RUNS; ++k) {
        const float s = half_bits_to_float(sb[k / L::kRunsPerGroup]);
        float x[L::LEN];
#pragma unroll
        for (int n = 0; n < L::LEN; ++n) {
            const int e = k * L::LEN + n;
            const int q = static_cast<int>((c[e * BITS / 32] >> (e * BITS % 32)) & ((1u << BITS) - 1u)) -
                          F::kZero;
            x[n] = s * static_cast<float>(q);
        }
        uint16_t *p = dst + L::dim(lane, k);
        if constexpr (VALUE) {
            *reinterpret_cast<uint32_t *>(p) = pack_bf2(x[0], x[1]);
        } else {
            st16(p, make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]),
                               pack_bf2(x[6], x[7])));
        }
    }
}

template <int D, int BITS>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(KvReadArgs a) {
    pdl_trigger();
    pdl_wait();
    if (blockIdx.y == 0)
        read_rows<D, BITS, false>(a);
    else
        read_rows<D, BITS, true>(a);
}

// ---- host ---------------------------------------------------------------------

// Blocks of a launch over `rows` token heads (value rows take the most lanes).
static dim3 row_grid(int64_t rows) {
    constexpr int64_t per_block = kKvThreads / 8;
    return dim3(static_cast<unsigned>((rows + per_block - 1) / per_block), 2);
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
    if (!rn::current_device_info()) return RN_ERR_DEVICE;
    rn::KvWriteArgs a;
    a.kv = qkv + static_cast<int64_t>(Hq) * D;
    a.stride = (static_cast<int64_t>(Hq) + 2 * static_cast<int64_t>(Hkv)) * D;
    a.slots = slots;
    a.T = T;
    a.cache = {codes, scales, num_pages, Hkv, rn::kv_log2_page(page_size)};
    a.num_slots = num_pages << a.cache.log2_page;
    return rn::kv_dispatch(D, format, [&](auto d, auto bits) {
        return rn::launch_pdl(rn::kv_write_kernel<d.value, bits.value>, rn::row_grid(T * Hkv),
                              dim3(rn::kKvThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
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
    if (!rn::current_device_info()) return RN_ERR_DEVICE;
    rn::KvReadArgs a;
    a.cache = {const_cast<uint8_t *>(codes), const_cast<uint16_t *>(scales), num_pages, Hkv,
               rn::kv_log2_page(page_size)};
    a.page_table = page_table;
    a.B = B;
    a.max_pages = max_pages;
    a.cu_lens = cu_lens;
    a.starts = starts;
    a.total = total;
    a.out[0] = k;
    a.out[1] = v;
    return rn::kv_dispatch(D, format, [&](auto d, auto bits) {
        return rn::launch_pdl(rn::kv_read_kernel<d.value, bits.value>, rn::row_grid(total * Hkv),
                              dim3(rn::kKvThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
    });
}

}  // extern "C"
