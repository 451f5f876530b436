// qk_axes.cu -- per-head Q/K RMSNorm + rotary positions with several axes, and its
// gradient (sm_103a).
//
// With n^ = x rstd, rstd = 1 / sqrt(mean x^2 + eps), R the rotation of every pair by the
// position of its own axis:
//   forward   o = R (n^ w)
//   gradient  g = R^T do,  dw = sum over tokens and heads of g n^,
//             u = g w,     dx = rstd (u - n^ mean(u n^))
// Both read every value once and write every value once: HBM bounds them.
//
// Lane layout: D / 16 lanes hold a head, each two runs of eight elements ("chunks"): lane
// l has chunk l and chunk l + D / 16, so that every load and store instruction of a head
// covers whole 128-byte lines whatever rotary_dim is.  Pairs (i, i + D/2) then lie in one
// lane; with a smaller rotary_dim the partner chunk is another lane's and comes by a
// shuffle of its packed words.  Neighbouring pairs lie in one lane anyway.
//
// A group of lanes takes one token and walks over a part of its heads, so a lane turns by
// the same angles throughout: cosines and sines are fetched once for each (token, part).
// Parts hold query heads or key heads only: one weight in registers, and in the gradient
// one set of 16 sums of dw a lane.
#include "rn_common.cuh"
#include "rn_host.h"

namespace rn {

// This translation unit's status word; rn_device_status() ORs it with the others'.
static __device__ unsigned int g_qk_axes_status = 0u;

constexpr int kMaxAxes = 4;

struct QkAxesArgs {
    const uint16_t *x;   // [T, >= (Hq + Hkv) D], rows x_stride apart
    int64_t x_stride;
    const uint16_t *dout;  // gradient only
    int64_t dout_stride;
    uint16_t *y;           // out, or dx
    int64_t y_stride;
    const uint16_t *wq;
    const uint16_t *wk;
    const void *cos_sin;
    const int64_t *pos;    // [axes, T], rows pos_stride apart
    int64_t pos_stride;
    int64_t max_pos;
    int64_t T;
    int Hq, Hkv;
    float eps;
    uint32_t pair_axis[8];  // two bits a pair
    uint8_t used;           // axes that turn some pair, a bit each
    bool table_bf16;
    int q_parts, k_parts;   // parts of a token's query and key heads
    // gradient: blocks 0 .. q_blocks - 1 take the query parts, the others the key parts,
    // and each leaves its sums of dw in row blockIdx.x of partial [blocks, D]
    int q_blocks;
    float *partial;
};

template <int D, int R, int STYLE>
struct AxesLane {
    static constexpr int LPH = D / 16;     // lanes of a head
    static constexpr int TOKENS = 32 / LPH;  // tokens of a warp
    static constexpr bool kWhole = R == D;
    static constexpr int kRotary = R / 8;    // R < D: lanes whose first chunk turns
    static constexpr int kPartner = R / 16;  // and, in neox pairs, how far its partner's lane is
};

// c[0..3], s[0..3]: cosines and sines of four pairs from p on, of a token at `pos`.
template <int R>
__device__ __forceinline__ void load_angles(const QkAxesArgs &a, const int64_t (&pos)[kMaxAxes], int p, float *c,
                                            float *s) {
    const uint32_t code = a.pair_axis[p >> 4] >> (2 * (p & 15)) & 0xFFu;
    const auto at = [&](uint32_t axis) {
        return axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
    };
    const int64_t row = at(code & 3u) * R + p;
    if (code == (code & 3u) * 0x55u) {  // one axis: one run of the table each
        if (a.table_bf16) {
            const uint16_t *t = static_cast<const uint16_t *>(a.cos_sin) + row;
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(t));
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(t + R / 2));
            c[0] = bf_lo(u.x); c[1] = bf_hi(u.x); c[2] = bf_lo(u.y); c[3] = bf_hi(u.y);
            s[0] = bf_lo(v.x); s[1] = bf_hi(v.x); s[2] = bf_lo(v.y); s[3] = bf_hi(v.y);
        } else {
            const float *t = static_cast<const float *>(a.cos_sin) + row;
            const float4 u = __ldg(reinterpret_cast<const float4 *>(t));
            const float4 v = __ldg(reinterpret_cast<const float4 *>(t + R / 2));
            c[0] = u.x; c[1] = u.y; c[2] = u.z; c[3] = u.w;
            s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = at(code >> (2 * i) & 3u) * R + p + i;
        if (a.table_bf16) {
            const uint16_t *t = static_cast<const uint16_t *>(a.cos_sin) + r;
            c[i] = bf_lo(__ldg(t));
            s[i] = bf_lo(__ldg(t + R / 2));
        } else {
            const float *t = static_cast<const float *>(a.cos_sin) + r;
            c[i] = __ldg(t);
            s[i] = __ldg(t + R / 2);
        }
    }
}

// The angles of a lane's elements (see turn()) for the token at t; false where one of its
// positions is outside the table.
template <int D, int R, int STYLE>
__device__ __forceinline__ bool lane_angles(const QkAxesArgs &a, int64_t t, int sub, float (&c)[8], float (&s)[8]) {
    using L = AxesLane<D, R, STYLE>;
    int64_t pos[kMaxAxes];
    bool ok = true;
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i) {
        pos[i] = 0;
        if (a.used >> i & 1) {
            pos[i] = __ldg(a.pos + i * a.pos_stride + t);
            if (static_cast<uint64_t>(pos[i]) >= static_cast<uint64_t>(a.max_pos)) {
                ok = false;
                pos[i] = 0;  // keeps every address in range; nothing is stored
            }
        }
    }
    if constexpr (L::kWhole && STYLE == RN_ROPE_NEOX) {
        load_angles<R>(a, pos, sub * 8, c, s);
        load_angles<R>(a, pos, sub * 8 + 4, c + 4, s + 4);
    } else if constexpr (L::kWhole) {
        load_angles<R>(a, pos, sub * 4, c, s);
        load_angles<R>(a, pos, (sub + L::LPH) * 4, c + 4, s + 4);
    } else if constexpr (STYLE == RN_ROPE_NEOX) {
        if (sub < L::kRotary) {
            const int p = (sub < L::kPartner ? sub : sub - L::kPartner) * 8;
            load_angles<R>(a, pos, p, c, s);
            load_angles<R>(a, pos, p + 4, c + 4, s + 4);
        }
        if (sub < L::kPartner)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = -s[e];
    } else {
        if (sub < L::kRotary) load_angles<R>(a, pos, sub * 4, c, s);
    }
    return ok;
}

// Turns a lane's elements lo, hi: by R, or with `back` by R^T.  `other`: the partner
// lane's first chunk where it is another's (neox pairs, R < D).
template <int D, int R, int STYLE>
__device__ __forceinline__ void turn(float (&lo)[8], float (&hi)[8], const float (&other)[8], const float (&c)[8],
                                     const float (&s)[8], int sub, bool back) {
    using L = AxesLane<D, R, STYLE>;
    const auto pair = [&](float &x, float &y, float co, float si) {
        const float b = back ? -si : si;
        const float u = x * co - y * b, v = y * co + x * b;
        x = u;
        y = v;
    };
    if constexpr (L::kWhole && STYLE == RN_ROPE_NEOX) {
#pragma unroll
        for (int e = 0; e < 8; ++e) pair(lo[e], hi[e], c[e], s[e]);
    } else if constexpr (STYLE == RN_ROPE_NEOX) {
        if (sub < L::kRotary)
#pragma unroll
            for (int e = 0; e < 8; ++e) lo[e] = lo[e] * c[e] + other[e] * (back ? -s[e] : s[e]);
    } else if (L::kWhole || sub < L::kRotary) {
#pragma unroll
        for (int i = 0; i < 4; ++i) pair(lo[2 * i], lo[2 * i + 1], c[i], s[i]);
        if constexpr (L::kWhole)
#pragma unroll
            for (int i = 0; i < 4; ++i) pair(hi[2 * i], hi[2 * i + 1], c[4 + i], s[4 + i]);
    }
}

template <class E>
__device__ __forceinline__ void widen(const uint4 &u, float (&x)[8]) {
    x[0] = E::lo(u.x); x[1] = E::hi(u.x); x[2] = E::lo(u.y); x[3] = E::hi(u.y);
    x[4] = E::lo(u.z); x[5] = E::hi(u.z); x[6] = E::lo(u.w); x[7] = E::hi(u.w);
}
template <class E>
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
    return make_uint4(E::pack(x[0], x[1]), E::pack(x[2], x[3]), E::pack(x[4], x[5]), E::pack(x[6], x[7]));
}
template <class E>
__device__ __forceinline__ float square_sum(const uint4 &u, float acc) {
    return E::sq_acc(E::sq_acc(E::sq_acc(E::sq_acc(acc, u.x), u.y), u.z), u.w);
}
__device__ __forceinline__ uint4 shuffle_xor(const uint4 &u, int lanes) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, u.x, lanes), __shfl_xor_sync(0xffffffffu, u.y, lanes),
                      __shfl_xor_sync(0xffffffffu, u.z, lanes), __shfl_xor_sync(0xffffffffu, u.w, lanes));
}

// The partner lane's chunk; lanes beyond the rotary ones take part and use nothing.
template <int D, int R, int STYLE>
__device__ __forceinline__ uint4 partner(const uint4 &u) {
    using L = AxesLane<D, R, STYLE>;
    if constexpr (!L::kWhole && STYLE == RN_ROPE_NEOX) return shuffle_xor(u, L::kPartner);
    return u;
}

constexpr int kAxesThreads = 256;
constexpr int kAxesWarps = kAxesThreads / 32;

// Heads h0 .. h1 - 1 of part `part` of n equal parts of `heads` heads.
__device__ __forceinline__ void part_heads(int part, int n, int heads, int &h0, int &h1) {
    h0 = static_cast<int>(static_cast<int64_t>(part) * heads / n);
    h1 = static_cast<int>(static_cast<int64_t>(part + 1) * heads / n);
}

constexpr int kFwdAhead = 4;  // heads whose loads are under way together

template <int D, int R, int STYLE, class E>
__global__ void __launch_bounds__(kAxesThreads) qk_axes_fwd_kernel(const __grid_constant__ QkAxesArgs a) {
    using L = AxesLane<D, R, STYLE>;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane % L::LPH;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kAxesWarps + (threadIdx.x >> 5);
    const int parts = a.q_parts + a.k_parts;
    const int64_t t = unit / parts * L::TOKENS + lane / L::LPH;
    const int part = static_cast<int>(unit % parts);
    if (unit / parts * L::TOKENS >= a.T) return;  // a whole warp
    const bool live = t < a.T;
    const bool is_q = part < a.q_parts;
    int h0, h1;
    if (is_q) {
        part_heads(part, a.q_parts, a.Hq, h0, h1);
    } else {
        part_heads(part - a.q_parts, a.k_parts, a.Hkv, h0, h1);
        h0 += a.Hq;
        h1 += a.Hq;
    }
    const uint16_t *row = a.x + t * a.x_stride + sub * 8;
    uint16_t *out = a.y + t * a.y_stride + sub * 8;
    constexpr int HI = D / 2;
    uint4 lo[kFwdAhead], hi[kFwdAhead];
    const auto fetch = [&](int h) {
#pragma unroll
        for (int u = 0; u < kFwdAhead; ++u) {
            lo[u] = hi[u] = make_uint4(0u, 0u, 0u, 0u);
            if (live && h + u < h1) {
                lo[u] = *reinterpret_cast<const uint4 *>(row + static_cast<int64_t>(h + u) * D);
                hi[u] = *reinterpret_cast<const uint4 *>(row + static_cast<int64_t>(h + u) * D + HI);
            }
        }
    };
    fetch(h0);
    // the heads' loads do not wait for the position and its angles
    const uint16_t *w = (is_q ? a.wq : a.wk) + sub * 8;
    const uint4 wl = ld_ro16(w), wh = ld_ro16(w + HI);
    const uint4 wp = partner<D, R, STYLE>(wl);
    float c[8], s[8];
    bool ok = false;
    if (live) {
        ok = lane_angles<D, R, STYLE>(a, t, sub, c, s);
        if (!ok && sub == 0) atomicOr(&g_qk_axes_status, RN_STATUS_BAD_POSITION);
    }
    for (int h = h0; h < h1; h += kFwdAhead) {
        if (h != h0) fetch(h);
        float rstd[kFwdAhead];
#pragma unroll
        for (int u = 0; u < kFwdAhead; ++u) rstd[u] = square_sum<E>(hi[u], square_sum<E>(lo[u], 0.0f));
#pragma unroll
        for (int u = 0; u < kFwdAhead; ++u)
            rstd[u] = __frsqrt_rn(group_sum<L::LPH>(rstd[u]) / static_cast<float>(D) + a.eps);
#pragma unroll
        for (int u = 0; u < kFwdAhead; ++u) {
            const uint4 po = partner<D, R, STYLE>(lo[u]);
            if (!ok || h + u >= h1) continue;  // (a group of lanes alike; nothing below crosses lanes)
            float x[8], y[8], o[8], wv[8];
            const auto weigh = [&](const uint4 &v, const uint4 &weight, float (&to)[8]) {
                widen<E>(v, to);
                widen<E>(weight, wv);
#pragma unroll
                for (int e = 0; e < 8; ++e) to[e] = to[e] * rstd[u] * wv[e];
            };
            weigh(lo[u], wl, x);
            weigh(hi[u], wh, y);
            if constexpr (!L::kWhole && STYLE == RN_ROPE_NEOX) weigh(po, wp, o);
            turn<D, R, STYLE>(x, y, o, c, s, sub, false);
            st16(out + static_cast<int64_t>(h + u) * D, narrow<E>(x));
            st16(out + static_cast<int64_t>(h + u) * D + HI, narrow<E>(y));
        }
    }
}

constexpr int kBwdAhead = 2;

template <int D, int R, int STYLE, class E>
__global__ void __launch_bounds__(kAxesThreads, 2) qk_axes_bwd_kernel(const __grid_constant__ QkAxesArgs a) {
    using L = AxesLane<D, R, STYLE>;
    constexpr int GROUPS = kAxesWarps * L::TOKENS;  // groups of lanes of the block
    __shared__ float sums[GROUPS][D];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, sub = lane % L::LPH;
    const bool is_q = static_cast<int>(blockIdx.x) < a.q_blocks;
    const int block = is_q ? blockIdx.x : blockIdx.x - a.q_blocks;
    const int blocks = is_q ? a.q_blocks : gridDim.x - a.q_blocks;
    const int parts = is_q ? a.q_parts : a.k_parts, heads = is_q ? a.Hq : a.Hkv, first = is_q ? 0 : a.Hq;
    const int64_t units = (a.T + L::TOKENS - 1) / L::TOKENS * parts;
    constexpr int HI = D / 2;
    const uint16_t *w = (is_q ? a.wq : a.wk) + sub * 8;
    const uint4 wl = ld_ro16(w), wh = ld_ro16(w + HI);
    float dl[8], dh[8];  // sums of g n^
#pragma unroll
    for (int e = 0; e < 8; ++e) dl[e] = dh[e] = 0.0f;

    for (int64_t unit = static_cast<int64_t>(block) * kAxesWarps + (threadIdx.x >> 5); unit < units;
         unit += static_cast<int64_t>(blocks) * kAxesWarps) {
        const int64_t t = unit / parts * L::TOKENS + lane / L::LPH;
        const bool live = t < a.T;
        int h0, h1;
        part_heads(static_cast<int>(unit % parts), parts, heads, h0, h1);
        h0 += first;
        h1 += first;
        const uint16_t *row = a.x + t * a.x_stride + sub * 8;
        const uint16_t *grad = a.dout + t * a.dout_stride + sub * 8;
        uint16_t *out = a.y + t * a.y_stride + sub * 8;
        uint4 xl[kBwdAhead], xh[kBwdAhead], gl[kBwdAhead], gh[kBwdAhead];
        const auto fetch = [&](int h) {
#pragma unroll
            for (int u = 0; u < kBwdAhead; ++u) {
                xl[u] = xh[u] = gl[u] = gh[u] = make_uint4(0u, 0u, 0u, 0u);
                if (live && h + u < h1) {
                    const int64_t at = static_cast<int64_t>(h + u) * D;
                    xl[u] = *reinterpret_cast<const uint4 *>(row + at);
                    xh[u] = *reinterpret_cast<const uint4 *>(row + at + HI);
                    gl[u] = *reinterpret_cast<const uint4 *>(grad + at);
                    gh[u] = *reinterpret_cast<const uint4 *>(grad + at + HI);
                }
            }
        };
        fetch(h0);
        float c[8], s[8];
        bool ok = false;
        if (live) {
            ok = lane_angles<D, R, STYLE>(a, t, sub, c, s);
            if (!ok && sub == 0) atomicOr(&g_qk_axes_status, RN_STATUS_BAD_POSITION);
        }
        for (int h = h0; h < h1; h += kBwdAhead) {
            if (h != h0) fetch(h);
            float rstd[kBwdAhead];
#pragma unroll
            for (int u = 0; u < kBwdAhead; ++u) rstd[u] = square_sum<E>(xh[u], square_sum<E>(xl[u], 0.0f));
#pragma unroll
            for (int u = 0; u < kBwdAhead; ++u)
                rstd[u] = __frsqrt_rn(group_sum<L::LPH>(rstd[u]) / static_cast<float>(D) + a.eps);
#pragma unroll
            for (int u = 0; u < kBwdAhead; ++u) {
                float x[8], y[8], p[8], q[8], o[8], wv[8];
                const uint4 po = partner<D, R, STYLE>(gl[u]);
                widen<E>(gl[u], p);
                widen<E>(gh[u], q);
                widen<E>(po, o);
                turn<D, R, STYLE>(p, q, o, c, s, sub, true);
                widen<E>(xl[u], x);
                widen<E>(xh[u], y);
                const bool use = ok && h + u < h1;
                float dot = 0.0f;
                // n^ = x rstd, dw += g n^, u = g w, dot = sum u n^
                widen<E>(wl, wv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= rstd[u];
                    if (use) dl[e] = fmaf(p[e], x[e], dl[e]);
                    p[e] *= wv[e];
                    dot = fmaf(p[e], x[e], dot);
                }
                widen<E>(wh, wv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[e] *= rstd[u];
                    if (use) dh[e] = fmaf(q[e], y[e], dh[e]);
                    q[e] *= wv[e];
                    dot = fmaf(q[e], y[e], dot);
                }
                dot = group_sum<L::LPH>(dot) / static_cast<float>(D);
                if (!use) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = rstd[u] * fmaf(-x[e], dot, p[e]);
                    q[e] = rstd[u] * fmaf(-y[e], dot, q[e]);
                }
                st16(out + static_cast<int64_t>(h + u) * D, narrow<E>(p));
                st16(out + static_cast<int64_t>(h + u) * D + HI, narrow<E>(q));
            }
        }
    }

    // the block's sums of dw, its groups in their order
    const int group = (threadIdx.x >> 5) * L::TOKENS + lane / L::LPH;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        sums[group][sub * 8 + e] = dl[e];
        sums[group][HI + sub * 8 + e] = dh[e];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kAxesThreads) {
        float v = 0.0f;
#pragma unroll 8
        for (int g = 0; g < GROUPS; ++g) v += sums[g][d];
        a.partial[static_cast<int64_t>(blockIdx.x) * D + d] = v;
    }
}

// dw[which] (+)= the blocks' sums, in their order.  blockIdx.x: 32 dimensions, y: query or key.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) qk_axes_sum_kernel(const float *partial, int q_blocks, int blocks,
                                                                     int D, float *dwq, float *dwk, int accumulate) {
    __shared__ float sums[kSumWarps][32];
    pdl_trigger();
    pdl_wait();
    float *dw = blockIdx.y == 0 ? dwq : dwk;
    if (!dw) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = blockIdx.x * 32 + lane;
    const int b0 = blockIdx.y == 0 ? 0 : q_blocks, b1 = blockIdx.y == 0 ? q_blocks : blocks;
    float v = 0.0f;
#pragma unroll 8
    for (int b = b0 + warp; b < b1; b += kSumWarps) v += partial[static_cast<int64_t>(b) * D + d];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0) {
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < kSumWarps; ++k) v += sums[k][lane];
        dw[d] = accumulate ? dw[d] + v : v;
    }
}

// ---- host -------------------------------------------------------------------------------

constexpr int kBwdBlocks = 4;  // blocks an SM, at most

static int64_t bwd_workspace(int sm_count, int D) {
    return static_cast<int64_t>(sm_count) * kBwdBlocks * D * 4;
}

// Parts that `heads` heads are cut into so that a part has up to `most` of them.
static int parts_of(int heads, int most) { return (heads + most - 1) / most; }

// Heads of a part: eight, or fewer where tokens are too few to fill the GPU's warps.
static int part_size(int64_t warps_of_tokens, int heads, int64_t want) {
    for (int n = 8; n > 1; n /= 2)
        if (warps_of_tokens * parts_of(heads, n) >= want) return n;
    return 1;
}

template <int D, int R, int STYLE, class E>
static int qk_axes_launch(QkAxesArgs &a, bool backward, float *dwq, float *dwk, int accumulate, const DeviceInfo &dev,
                          cudaStream_t st) {
    using L = AxesLane<D, R, STYLE>;
    const int64_t quads = (a.T + L::TOKENS - 1) / L::TOKENS;
    const int n = part_size(quads, a.Hq + a.Hkv, static_cast<int64_t>(dev.sm_count) * 16);
    a.q_parts = parts_of(a.Hq, n);
    a.k_parts = parts_of(a.Hkv, n);
    const int64_t units = quads * (a.q_parts + a.k_parts);
    if (!backward) {
        const int64_t blocks = (units + kAxesWarps - 1) / kAxesWarps;
        return launch_pdl(qk_axes_fwd_kernel<D, R, STYLE, E>, dim3(static_cast<unsigned>(blocks)), dim3(kAxesThreads),
                          0, st, a);
    }
    const int64_t most = static_cast<int64_t>(dev.sm_count) * 2;
    const auto blocks_of = [&](int64_t u, int64_t cap) {
        const int64_t b = (u + kAxesWarps - 1) / kAxesWarps;
        return static_cast<int>(b < cap ? b : cap);
    };
    // shares of the grid by their heads
    int64_t q_cap = most * a.Hq / (a.Hq + a.Hkv);
    if (q_cap < 1) q_cap = 1;
    if (q_cap > most - 1) q_cap = most - 1;
    a.q_blocks = blocks_of(quads * a.q_parts, a.Hkv ? q_cap : most);
    const int k_blocks = blocks_of(quads * a.k_parts, a.Hq ? most - q_cap : most);
    const int blocks = a.q_blocks + k_blocks;
    const int rc = launch_pdl(qk_axes_bwd_kernel<D, R, STYLE, E>, dim3(static_cast<unsigned>(blocks)),
                              dim3(kAxesThreads), 0, st, a);
    if (rc != RN_OK || (!dwq && !dwk)) return rc;
    return launch_pdl(qk_axes_sum_kernel, dim3(D / 32, 2), dim3(32 * kSumWarps), 0, st,
                      static_cast<const float *>(a.partial), a.q_blocks, blocks, D, dwq, dwk, accumulate);
}

template <int STYLE, class E>
static int qk_axes_layout(QkAxesArgs &a, int D, int r, bool backward, float *dwq, float *dwk, int accumulate,
                          const DeviceInfo &dev, cudaStream_t st) {
#define RN_AXES_GO(D_, R_) \
    if (D == (D_) && r == (R_)) return qk_axes_launch<D_, R_, STYLE, E>(a, backward, dwq, dwk, accumulate, dev, st);
    RN_AXES_GO(64, 64) RN_AXES_GO(64, 32) RN_AXES_GO(64, 16)
    RN_AXES_GO(128, 128) RN_AXES_GO(128, 64) RN_AXES_GO(128, 32)
    RN_AXES_GO(256, 256) RN_AXES_GO(256, 128) RN_AXES_GO(256, 64)
#undef RN_AXES_GO
    return RN_ERR_SHAPE;
}

struct QkAxesCall {
    int dtype, table_bf16, num_axes, D, rotary_dim, rope_style;
    const uint8_t *pair_axis;
    bool backward;
    float *dwq, *dwk;
    int accumulate;
    int64_t workspace_bytes;
};

static int qk_axes_run(QkAxesArgs &a, const QkAxesCall &k, rn_stream_t stream) {
    if (k.dtype != RN_DTYPE_BF16 && k.dtype != RN_DTYPE_F16) return RN_ERR_ARG;
    if (k.rope_style != RN_ROPE_NEOX && k.rope_style != RN_ROPE_GPTJ) return RN_ERR_ARG;
    if ((k.table_bf16 & ~1) || (k.accumulate & ~1)) return RN_ERR_ARG;
    const int D = k.D, r = k.rotary_dim;
    if (a.T < 0 || a.Hq < 0 || a.Hkv < 0) return RN_ERR_SHAPE;
    if (D != 64 && D != 128 && D != 256) return RN_ERR_SHAPE;
    if (r != D && r != D / 2 && r != D / 4) return RN_ERR_SHAPE;
    if (k.num_axes < 1 || k.num_axes > kMaxAxes) return RN_ERR_SHAPE;
    const int64_t H = static_cast<int64_t>(a.Hq) + a.Hkv;
    if (H > INT32_MAX || (H > 0 && a.T > INT32_MAX / H)) return RN_ERR_SHAPE;
    if (a.max_pos < 1) return RN_ERR_SHAPE;
    const int64_t width = H * D;
    const auto bad_stride = [&](int64_t stride) { return width > 0 && a.T > 1 && (stride < width || stride % 8 != 0); };
    if (bad_stride(a.x_stride) || bad_stride(a.y_stride) || (k.backward && bad_stride(a.dout_stride)))
        return RN_ERR_SHAPE;
    if (a.pos_stride < 0 || (k.num_axes > 1 && a.pos_stride != 0 && a.pos_stride < a.T)) return RN_ERR_SHAPE;
    if (!k.pair_axis) return RN_ERR_NULL;
    a.used = 0;
    for (uint32_t &v : a.pair_axis) v = 0;
    for (int i = 0; i < r / 2; ++i) {
        if (k.pair_axis[i] >= k.num_axes) return RN_ERR_ARG;
        a.used |= static_cast<uint8_t>(1u << k.pair_axis[i]);
        a.pair_axis[i >> 4] |= static_cast<uint32_t>(k.pair_axis[i]) << (2 * (i & 15));
    }
    const bool empty = a.T == 0 || H == 0;
    const bool weights = k.backward && (k.dwq || k.dwk);
    if (empty && !weights) return RN_OK;
    if (!empty) {
        if (!a.x || !a.y || !a.wq || !a.wk || !a.cos_sin || !a.pos) return RN_ERR_NULL;
        if (k.backward && (!a.dout || !a.partial)) return RN_ERR_NULL;
    }
    if (!aligned16(a.x) || !aligned16(a.y) || !aligned16(a.wq) || !aligned16(a.wk) || !aligned16(a.cos_sin) ||
        !aligned16(a.dout) || !aligned16(a.partial) || (reinterpret_cast<uintptr_t>(a.pos) & 7u) ||
        ((reinterpret_cast<uintptr_t>(k.dwq) | reinterpret_cast<uintptr_t>(k.dwk)) & 3u))
        return RN_ERR_ALIGN;
    if (k.backward && k.dwq && k.dwq == k.dwk) return RN_ERR_ARG;
    const DeviceInfo *dev = current_device_info();
    if (!dev) return RN_ERR_DEVICE;
    const auto st = reinterpret_cast<cudaStream_t>(stream);
    if (empty)  // no token: sums of nothing
        return launch_pdl(qk_axes_sum_kernel, dim3(static_cast<unsigned>(D / 32), 2), dim3(32 * kSumWarps), 0, st,
                          static_cast<const float *>(nullptr), 0, 0, D, k.dwq, k.dwk, k.accumulate);
    if (k.backward && k.workspace_bytes < bwd_workspace(dev->sm_count, D)) return RN_ERR_ARG;
    a.table_bf16 = k.table_bf16 != 0;
#define RN_AXES_FORMAT(S_, E_) \
    return qk_axes_layout<S_, E_>(a, D, r, k.backward, k.dwq, k.dwk, k.accumulate, *dev, st)
    if (k.rope_style == RN_ROPE_GPTJ) {
        if (k.dtype == RN_DTYPE_F16) RN_AXES_FORMAT(RN_ROPE_GPTJ, F16);
        RN_AXES_FORMAT(RN_ROPE_GPTJ, Bf16);
    }
    if (k.dtype == RN_DTYPE_F16) RN_AXES_FORMAT(RN_ROPE_NEOX, F16);
    RN_AXES_FORMAT(RN_ROPE_NEOX, Bf16);
#undef RN_AXES_FORMAT
}

int qk_axes_status(unsigned int *out, int clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_qk_axes_status, sizeof v) != cudaSuccess) {
        cudaGetLastError();
        return RN_ERR_DEVICE;
    }
    if (clear && v != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_qk_axes_status, &zero, sizeof zero) != cudaSuccess) {
            cudaGetLastError();
            return RN_ERR_DEVICE;
        }
    }
    *out = v;
    return RN_OK;
}

}  // namespace rn

extern "C" {

int qk_norm_rope_axes_fwd(int dtype, const void *qkv, int64_t qkv_stride, const void *wq, const void *wk,
                          const void *cos_sin, int table_bf16, int64_t max_pos, const int64_t *positions,
                          int64_t pos_stride, const uint8_t *pair_axis, int num_axes, int64_t T, int Hq, int Hkv, int D,
                          int rotary_dim, float eps, int rope_style, void *out, int64_t out_stride,
                          rn_stream_t stream) {
    rn::QkAxesArgs a = {};
    a.x = static_cast<const uint16_t *>(qkv);
    a.x_stride = qkv_stride;
    a.y = static_cast<uint16_t *>(out);
    a.y_stride = out_stride;
    a.wq = static_cast<const uint16_t *>(wq);
    a.wk = static_cast<const uint16_t *>(wk);
    a.cos_sin = cos_sin;
    a.pos = positions;
    a.pos_stride = pos_stride;
    a.max_pos = max_pos;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.eps = eps;
    const rn::QkAxesCall k = {dtype,     table_bf16, num_axes, D,       rotary_dim, rope_style,
                              pair_axis, false,      nullptr,  nullptr, 0,          0};
    return rn::qk_axes_run(a, k, stream);
}

int64_t qk_norm_rope_axes_workspace_bytes(int D) {
    if (D != 64 && D != 128 && D != 256) return RN_ERR_SHAPE;
    const rn::DeviceInfo *dev = rn::current_device_info();
    if (!dev) return RN_ERR_DEVICE;
    return rn::bwd_workspace(dev->sm_count, D);
}

int qk_norm_rope_axes_bwd(int dtype, const void *dout, int64_t dout_stride, const void *qkv, int64_t qkv_stride,
                          const void *wq, const void *wk, const void *cos_sin, int table_bf16, int64_t max_pos,
                          const int64_t *positions, int64_t pos_stride, const uint8_t *pair_axis, int num_axes,
                          int64_t T, int Hq, int Hkv, int D, int rotary_dim, float eps, int rope_style, void *dx,
                          int64_t dx_stride, float *dwq, float *dwk, int accumulate, void *workspace,
                          int64_t workspace_bytes, rn_stream_t stream) {
    rn::QkAxesArgs a = {};
    a.x = static_cast<const uint16_t *>(qkv);
    a.x_stride = qkv_stride;
    a.dout = static_cast<const uint16_t *>(dout);
    a.dout_stride = dout_stride;
    a.y = static_cast<uint16_t *>(dx);
    a.y_stride = dx_stride;
    a.wq = static_cast<const uint16_t *>(wq);
    a.wk = static_cast<const uint16_t *>(wk);
    a.cos_sin = cos_sin;
    a.pos = positions;
    a.pos_stride = pos_stride;
    a.max_pos = max_pos;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.eps = eps;
    a.partial = static_cast<float *>(workspace);
    const rn::QkAxesCall k = {dtype,     table_bf16, num_axes, D,   rotary_dim, rope_style,
                              pair_axis, true,       dwq,      dwk, accumulate, workspace_bytes};
    return rn::qk_axes_run(a, k, stream);
}

}  // extern "C"
