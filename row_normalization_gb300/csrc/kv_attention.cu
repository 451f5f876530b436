// kv_attention.cu -- causal attention of ragged queries over the quantised
// key/value cache (sm_103a).
//
// The simple form: one CTA for one query token and head.  Its warps take the
// visible tokens in turn, a lane the elements it finds in its share of the
// stored row; each warp keeps the running maximum and sum of its own tokens'
// softmax, and the four partial results are joined at the end.
#include "kv_common.cuh"

namespace rn {

static __device__ unsigned int g_kv_attention_status = 0u;

struct KvAttnArgs {
    const uint16_t *q;
    int64_t q_stride;
    KvCache cache;
    const int32_t *page_table;
    int64_t B;
    int64_t max_pages;
    const int32_t *kv_lens;
    const int64_t *cu_q;
    int64_t T;
    int64_t max_q_len;
    int Hq;
    float scale_log2;  // softmax scale * log2(e)
    int64_t window;
    int64_t sinks;
    uint16_t *out;
    float *lse;
};

constexpr int kAttnThreads = 128;

template <int D, int BITS>
__global__ void __launch_bounds__(kAttnThreads) kv_attention_simple_kernel(KvAttnArgs a) {
    using F = KvFormat<D, BITS>;
    constexpr int E = D / 32;  // stored elements a lane
    pdl_trigger();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t b = t, first = t, n = 1;
    if (a.cu_q) {
        if (t < a.cu_q[0] || t >= a.cu_q[a.B]) return;
        int64_t lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (a.cu_q[mid] <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        b = lo;
        first = a.cu_q[b];
        n = a.cu_q[b + 1] - first;
    }
    int64_t len = a.kv_lens[b];
    const int64_t room = a.max_pages << a.cache.log2_page;
    if (len > room || t - first >= a.max_q_len) {
        if (threadIdx.x == 0) atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
        if (t - first >= a.max_q_len) return;
        len = room;
    }
    const int64_t pos = len - n + (t - first);
    const int kvh = h / (a.Hq / a.cache.Hkv);
    // the lane's elements of the query in the order of the stored keys
    float q[E], o[E], m = -INFINITY, l = 0.0f;
    int kdim[E], vdim[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int e = lane * E + i;
        const int j = e / (F::kGroups * 8), g = e / 8 % F::kGroups;
        kdim[i] = 32 * g + 8 * j + e % 8;
        const int r = e / (D / 8), bb = e / 2 % (D / 16);
        vdim[i] = 16 * bb + 2 * r + e % 2;
        q[i] = bf_lo(a.q[t * a.q_stride + static_cast<int64_t>(h) * D + kdim[i]]) * a.scale_log2;
        o[i] = 0.0f;
    }
    for (int64_t j = warp; j <= pos; j += kAttnThreads / 32) {
        if (a.window && j <= pos - a.window && j >= a.sinks) {
            const int64_t lo = pos - a.window + 1;  // the window's first token
            j += (lo - j) / (kAttnThreads / 32) * (kAttnThreads / 32);
            if (j < lo) continue;
        }
        const int64_t page = a.page_table[b * a.max_pages + (j >> a.cache.log2_page)];
        const bool good = page >= 0 && page < a.cache.num_pages;
        if (!good && lane == 0) atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
        const int off = static_cast<int>(j & ((1 << a.cache.log2_page) - 1));
        float s = 0.0f;
        float vals[2][E];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int64_t r = good ? a.cache.row(page, which, kvh, off) : 0;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int e = lane * E + i;
                int c = 0;
                float sc = 0.0f;
                if (good) {
                    c = a.cache.codes[r * F::kRow + e * BITS / 8];
                    if (BITS == 4) c = c >> (4 * (e & 1)) & 15;
                    sc = half_bits_to_float(
                        a.cache.scales[r * F::kGroups + (which ? vdim[i] : kdim[i]) / 32]);
                }
                vals[which][i] = sc * static_cast<float>(c - F::kZero);
            }
        }
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(q[i], vals[0][i], s);
        s = warp_sum(s);
        const float mn = fmaxf(m, s);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float f = exp2f(m - base), p = exp2f(s - base);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = fmaf(p, vals[1][i], o[i] * f);
        m = mn;
    }
    __shared__ float sm_m[kAttnThreads / 32], sm_l[kAttnThreads / 32];
    __shared__ float sm_o[kAttnThreads / 32][D];
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) sm_o[warp][vdim[i]] = o[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.0f;
    for (int k = 0; k < kAttnThreads / 32; ++k) mm = fmaxf(mm, sm_m[k]);
    const float base = mm == -INFINITY ? 0.0f : mm;
    float f[kAttnThreads / 32];
    for (int k = 0; k < kAttnThreads / 32; ++k) {
        f[k] = exp2f(sm_m[k] - base);
        ll += sm_l[k] * f[k];
    }
    for (int d = threadIdx.x; d < D; d += kAttnThreads) {
        float x = 0.0f;
        for (int k = 0; k < kAttnThreads / 32; ++k) x = fmaf(sm_o[k][d], f[k], x);
        x = ll == 0.0f ? 0.0f : x / ll;
        a.out[(t * a.Hq + h) * D + d] = static_cast<uint16_t>(pack_bf2(x, 0.0f));
    }
    if (threadIdx.x == 0 && a.lse)
        a.lse[t * a.Hq + h] = ll == 0.0f ? -INFINITY : base * 0.6931471805599453f + logf(ll);
}

int kv_attention_status(unsigned int *out, int clear) {
    return kv_status_word(g_kv_attention_status, out, clear);
}

template <int D, int BITS>
static int kv_attention_launch(const KvAttnArgs &a, cudaStream_t st) {
    return launch_pdl(kv_attention_simple_kernel<D, BITS>,
                      dim3(static_cast<unsigned>(a.T), static_cast<unsigned>(a.Hq)),
                      dim3(kAttnThreads), 0, st, a);
}

static int kv_attention_check(int format, int64_t B, int Hq, int Hkv, int D, int64_t max_q_len) {
    const int rc = kv_check_sizes(format, Hkv, D, 16, 1);
    if (rc != RN_OK) return rc;
    if (Hq < 1 || Hq > 65535 || Hq % Hkv != 0) return RN_ERR_SHAPE;
    if (B < 0 || B > INT32_MAX / Hq || max_q_len < 0 || max_q_len > INT32_MAX / Hq) return RN_ERR_SHAPE;
    return RN_OK;
}

}  // namespace rn

extern "C" {

int64_t kv_attention_workspace_bytes(int format, int64_t B, int Hq, int Hkv, int D,
                                     int64_t max_q_len) {
    const int rc = rn::kv_attention_check(format, B, Hq, Hkv, D, max_q_len);
    if (rc != RN_OK) return rc;
    return 16;
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
    if (workspace_bytes < kv_attention_workspace_bytes(format, B, Hq, Hkv, D, max_q_len))
        return RN_ERR_ARG;
    if (!rn::current_device_info()) return RN_ERR_DEVICE;
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
    a.window = window;
    a.sinks = sinks;
    a.out = out;
    a.lse = lse;
    return rn::kv_dispatch(D, format, [&](auto d, auto bits) {
        return rn::kv_attention_launch<d.value, bits.value>(a, reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
