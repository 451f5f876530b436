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
// the same angles throughout: cosines and sines are fetched once for each (token, part), and
// the weights multiplied into them in the forward pass.  Parts hold query heads or key heads
// only: one weight in registers, and in the gradient one set of 16 sums of dw a lane.
// Every lane copies its own elements ahead into its own places in shared memory.  That beats
// loads into registers (16384 tokens of 40 heads of 128, us): forward 65.3 -> 55.2, of which the
// bytes need 50.8; gradient 99.5 -> 80.9, of 75.5.  Three stages are enough for the forward pass:
// 24 warps an SM with two heads of 1 KB under way each; eight stages took 56.9 there and 18.9
// against 16.5 at 4096 tokens, as a warp begins later.
//
// What is left: a quarter of the gradient at 4096 tokens (27.9 us, floor 18.9) is its second
// launch, beginning and end; axes that change within four pairs cost 4 to 20% (heads of 256 that
// turn a half of 128 by three interleaved axes: 57.9 us forward, 96.9 gradient, floors as above).
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
    int part_heads;         // heads of a part, but for the last
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

// A token's positions on the axes that turn some pair; false where one is outside the table.
struct Positions {
    int at[kMaxAxes];
    bool ok;

    __device__ __forceinline__ void load(const QkAxesArgs &a, int64_t t, bool live) {
        ok = live;
#pragma unroll
        for (int i = 0; i < kMaxAxes; ++i) {
            at[i] = 0;
            if (live && (a.used >> i & 1)) {
                const int64_t p = __ldg(a.pos + i * a.pos_stride + t);
                const bool in = static_cast<uint64_t>(p) < static_cast<uint64_t>(a.max_pos);
                ok &= in;
                at[i] = in ? static_cast<int>(p) : 0;  // keeps every address in range; nothing is stored
            }
        }
    }
};

// c[0..3], s[0..3]: cosines and sines of four pairs from p on, of a token at `pos`.
template <int R>
__device__ __forceinline__ void load_angles(const QkAxesArgs &a, const Positions &pos, int p, float *c, float *s) {
    const uint32_t code = a.pair_axis[p >> 4] >> (2 * (p & 15)) & 0xFFu;
    const auto at = [&](uint32_t axis) -> int64_t {
        return axis == 0 ? pos.at[0] : axis == 1 ? pos.at[1] : axis == 2 ? pos.at[2] : pos.at[3];
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

// The angles of a lane's elements (see Turn) for a token at pos.
template <int D, int R, int STYLE>
__device__ __forceinline__ void lane_angles(const QkAxesArgs &a, const Positions &pos, int sub, float (&c)[8],
                                            float (&s)[8]) {
    using L = AxesLane<D, R, STYLE>;
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
}

// ---- a lane's elements -------------------------------------------------------------------

// Eight elements as they are stored, and as four fp32 pairs of neighbours.
template <class E>
__device__ __forceinline__ void widen(const uint4 &u, Pair (&x)[4]) {
    x[0] = Pair::of(E::lo(u.x), E::hi(u.x));
    x[1] = Pair::of(E::lo(u.y), E::hi(u.y));
    x[2] = Pair::of(E::lo(u.z), E::hi(u.z));
    x[3] = Pair::of(E::lo(u.w), E::hi(u.w));
}
template <class E>
__device__ __forceinline__ uint4 narrow(const Pair (&x)[4]) {
    return make_uint4(E::pack(x[0].v.x, x[0].v.y), E::pack(x[1].v.x, x[1].v.y), E::pack(x[2].v.x, x[2].v.y),
                      E::pack(x[3].v.x, x[3].v.y));
}
template <class E>
__device__ __forceinline__ float square_sum(const uint4 &u, float acc) {
    return E::sq_acc(E::sq_acc(E::sq_acc(E::sq_acc(acc, u.x), u.y), u.z), u.w);
}

// The partner lane's chunk; zeros for a lane that does not turn.  (All lanes take part.)
template <int D, int R, int STYLE>
__device__ __forceinline__ uint4 partner(const uint4 &u, int sub) {
    using L = AxesLane<D, R, STYLE>;
    if constexpr (L::kWhole || STYLE != RN_ROPE_NEOX) return u;
    const uint4 v = make_uint4(
        __shfl_xor_sync(0xffffffffu, u.x, L::kPartner), __shfl_xor_sync(0xffffffffu, u.y, L::kPartner),
        __shfl_xor_sync(0xffffffffu, u.z, L::kPartner), __shfl_xor_sync(0xffffffffu, u.w, L::kPartner));
    return sub < L::kRotary ? v : make_uint4(0u, 0u, 0u, 0u);
}

// What a lane multiplies its elements by: with x = lo, hi and o the partner's chunk,
//   neox, whole head:  lo' = lo a - hi b,  hi' = hi c + lo d   (pairs of neighbours at a time)
//   neox, a part:      lo' = lo a + o b,   hi' = hi c
//   neighbours:        of each pair (x, y) of a chunk: x' = x a.x - y a.y,  y' = y b.x + x b.y;
//                      a, b for lo, c, d for hi (which only weighs where it does not turn)
// The weights are in them: R w for the forward pass.
template <int D, int R, int STYLE>
struct Turn {
    using L = AxesLane<D, R, STYLE>;
    Pair a[4], b[4], c[4], d[4];

    // co, si as lane_angles gives them; wl, wh: weights; wo: the partner's
    __device__ __forceinline__ void set(const float (&co)[8], const float (&si)[8], const Pair (&wl)[4],
                                        const Pair (&wh)[4], const Pair (&wo)[4], int sub) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair cc = Pair::of(co[2 * i], co[2 * i + 1]), ss = Pair::of(si[2 * i], si[2 * i + 1]);
            if constexpr (STYLE == RN_ROPE_NEOX && L::kWhole) {
                a[i] = wl[i] * cc;
                b[i] = -(wh[i] * ss);
                c[i] = wh[i] * cc;
                d[i] = wl[i] * ss;
            } else if constexpr (STYLE == RN_ROPE_NEOX) {
                a[i] = sub < L::kRotary ? wl[i] * cc : wl[i];
                b[i] = wo[i] * ss;
                c[i] = wh[i];
            } else {
                const bool turns = L::kWhole || sub < L::kRotary;
                const float x = turns ? co[i] : 1.0f, y = turns ? si[i] : 0.0f;
                a[i] = Pair::of(wl[i].v.x * x, -wl[i].v.y * y);
                b[i] = Pair::of(wl[i].v.y * x, wl[i].v.x * y);
                const float p = L::kWhole ? co[4 + i] : 1.0f, q = L::kWhole ? si[4 + i] : 0.0f;
                c[i] = Pair::of(wh[i].v.x * p, -wh[i].v.y * q);
                d[i] = Pair::of(wh[i].v.y * p, wh[i].v.x * q);
            }
        }
    }
    __device__ __forceinline__ void apply(Pair (&lo)[4], Pair (&hi)[4], const Pair (&o)[4], int sub) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair x = lo[i], y = hi[i];
            if constexpr (STYLE == RN_ROPE_NEOX && L::kWhole) {
                lo[i] = x.fma(a[i], y * b[i]);
                hi[i] = y.fma(c[i], x * d[i]);
            } else if constexpr (STYLE == RN_ROPE_NEOX) {
                lo[i] = x.fma(a[i], o[i] * b[i]);
                hi[i] = y * c[i];
            } else {
                // (a lane that does not turn: a product with zero would make an infinity NaN)
                const float2 v = x.v, w = y.v;
                const bool turns = L::kWhole || sub < L::kRotary;
                lo[i] = Pair::of(fmaf(v.x, a[i].v.x, turns ? v.y * a[i].v.y : 0.0f),
                                 fmaf(v.y, b[i].v.x, turns ? v.x * b[i].v.y : 0.0f));
                hi[i] = L::kWhole ? Pair::of(fmaf(w.x, c[i].v.x, w.y * c[i].v.y), fmaf(w.y, d[i].v.x, w.x * d[i].v.y))
                                  : Pair::of(w.x * c[i].v.x, w.y * d[i].v.x);
            }
        }
    }
};

// ---- the stream of heads -----------------------------------------------------------------

// A unit is a part of the heads of a warp's tokens: part_heads query heads or key heads, or
// what is left of them.  A warp takes its units one after another as one stream of heads,
// each lane with its own elements, copied to its own places in shared memory some heads
// ahead: nothing waits for another lane, and the next unit comes in while one ends.  This is
// a place in the stream.
template <int TOKENS>
struct HeadPlace {
    int64_t t;            // the lanes' token
    int64_t quad, quads;  // of how many groups of TOKENS tokens
    int part, parts;      // parts first .. first + parts - 1 of a token's q_parts + k_parts
    int quad_step, part_step;
    int h, h1;            // the head, and the unit's end
    bool is_q, live;

    // Place `unit` of every `step`-th.
    __device__ __forceinline__ HeadPlace(const QkAxesArgs &a, int first, int parts_, uint32_t unit, uint32_t step)
        : quads((a.T + TOKENS - 1) / TOKENS), parts(first + parts_) {
        const uint32_t n = parts_;
        quad = unit / n;
        part = first + static_cast<int>(unit - static_cast<uint32_t>(quad) * n);
        quad_step = static_cast<int>(step / n);
        part_step = static_cast<int>(step - quad_step * n);
        enter(a);
    }
    __device__ __forceinline__ bool inside() const { return quad < quads; }
    __device__ __forceinline__ void enter(const QkAxesArgs &a) {
        t = quad * TOKENS + (threadIdx.x & 31) / (32 / TOKENS);
        live = t < a.T;  // (also where there is no such unit)
        is_q = part < a.q_parts;
        h = (is_q ? part : part - a.q_parts) * a.part_heads;
        h1 = min(h + a.part_heads, is_q ? a.Hq : a.Hkv);
        if (!is_q) {
            h += a.Hq;
            h1 += a.Hq;
        }
    }
    __device__ __forceinline__ void next_unit(const QkAxesArgs &a, int first) {
        quad += quad_step;
        part += part_step;
        if (part >= parts) {
            part -= parts - first;
            ++quad;
        }
        enter(a);
    }
    // On to the next head; true where a unit ends.
    __device__ __forceinline__ bool next(const QkAxesArgs &a, int first) {
        if (++h < h1) return false;
        next_unit(a, first);
        return true;
    }
};

// ---- forward ---------------------------------------------------------------------------

constexpr int kFwdThreads = 256;
constexpr int kFwdWarps = kFwdThreads / 32;
constexpr int kFwdBlocks = 3;   // blocks of an SM
constexpr int kFwdStages = 3;   // heads that a warp has under way or is taking

template <int D, int R, int STYLE, class E>
__global__ void __launch_bounds__(kFwdThreads, kFwdBlocks)
    qk_axes_fwd_kernel(const __grid_constant__ QkAxesArgs a) {
    using L = AxesLane<D, R, STYLE>;
    constexpr int HI = D / 2;
    extern __shared__ __align__(16) uint4 heads_in[];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L::LPH;
    HeadPlace<L::TOKENS> now(a, 0, a.q_parts + a.k_parts, blockIdx.x * kFwdWarps + warp, gridDim.x * kFwdWarps);
    HeadPlace<L::TOKENS> ahead = now;
    uint4 *in = heads_in + warp * (kFwdStages * 64) + lane;
    uint32_t head = 0, tail = 0;  // stages of the head to be copied next, and to be taken next
    const auto copy = [&] {
        if (ahead.live) {
            const uint16_t *x = a.x + ahead.t * a.x_stride + static_cast<int64_t>(ahead.h) * D + sub * 8;
            copy_async16(in + head * 64, x);
            copy_async16(in + head * 64 + 32, x + HI);
        }
        copy_commit();
        head = head + 1 == kFwdStages ? 0 : head + 1;
        ahead.next(a, 0);
    };
    Positions pos;
    pos.load(a, now.t, now.live);
#pragma unroll 1
    for (int i = 0; i < kFwdStages - 1; ++i) copy();

    while (now.inside()) {
        Turn<D, R, STYLE> turn;
        const bool ok = pos.ok;
        if (now.live && !ok && sub == 0) atomicOr(&g_qk_axes_status, RN_STATUS_BAD_POSITION);
        {
            const uint16_t *w = (now.is_q ? a.wq : a.wk) + sub * 8;
            const uint4 ul = ld_ro16(w), uh = ld_ro16(w + HI);
            Pair wl[4], wh[4], wo[4];
            float c[8] = {}, s[8] = {};
            if (ok) lane_angles<D, R, STYLE>(a, pos, sub, c, s);
            widen<E>(ul, wl);
            widen<E>(uh, wh);
            widen<E>(partner<D, R, STYLE>(ul, sub), wo);
            turn.set(c, s, wl, wh, wo, sub);
        }
        {
            HeadPlace<L::TOKENS> then = now;  // the next unit's positions come meanwhile
            then.next_unit(a, 0);
            pos.load(a, then.t, then.live);
        }
        bool end;
        do {
            copy_wait<kFwdStages - 2>();
            const uint4 lo = ld_shared16(in + tail * 64), hi = ld_shared16(in + tail * 64 + 32);
            tail = tail + 1 == kFwdStages ? 0 : tail + 1;
            copy();  // (to the stage that the head before came from)
            const float rstd = __frsqrt_rn(
                group_sum<L::LPH>(square_sum<E>(hi, square_sum<E>(lo, 0.0f))) / static_cast<float>(D) + a.eps);
            const uint4 po = partner<D, R, STYLE>(lo, sub);
            if (ok) {
                Pair x[4], y[4], o[4];
                widen<E>(lo, x);
                widen<E>(hi, y);
                widen<E>(po, o);
                const Pair r = Pair::both(rstd);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = x[i] * r;
                    y[i] = y[i] * r;
                    if constexpr (!L::kWhole && STYLE == RN_ROPE_NEOX) o[i] = o[i] * r;
                }
                turn.apply(x, y, o, sub);
                uint16_t *out = a.y + now.t * a.y_stride + static_cast<int64_t>(now.h) * D + sub * 8;
                st16(out, narrow<E>(x));
                st16(out + HI, narrow<E>(y));
            }
            end = now.next(a, 0);
        } while (!end);
    }
}

// ---- gradient ----------------------------------------------------------------------------

constexpr int kBwdThreads = 256;
constexpr int kBwdWarps = kBwdThreads / 32;
constexpr int kBwdBlocks = 2;  // blocks of an SM
constexpr int kBwdStages = 3;  // heads that a warp has under way or is taking

template <int D, int R, int STYLE, class E>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks)
    qk_axes_bwd_kernel(const __grid_constant__ QkAxesArgs a) {
    using L = AxesLane<D, R, STYLE>;
    constexpr int HI = D / 2;
    constexpr int GROUPS = kBwdWarps * L::TOKENS;  // groups of lanes of the block
    static_assert(GROUPS * D * 4 <= kBwdWarps * kBwdStages * 2048, "the sums take the place of the stages");
    extern __shared__ __align__(16) uint4 heads_in[];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L::LPH;
    // query heads or key heads alone
    const bool is_q = static_cast<int>(blockIdx.x) < a.q_blocks;
    const int block = is_q ? blockIdx.x : blockIdx.x - a.q_blocks;
    const int blocks = is_q ? a.q_blocks : gridDim.x - a.q_blocks;
    const int first = is_q ? 0 : a.q_parts;
    HeadPlace<L::TOKENS> now(a, first, is_q ? a.q_parts : a.k_parts, block * kBwdWarps + warp, blocks * kBwdWarps);
    HeadPlace<L::TOKENS> ahead = now;
    uint4 *in = heads_in + warp * (kBwdStages * 128) + lane;
    uint32_t head = 0, tail = 0;  // stages of the head to be copied next, and to be taken next
    const auto copy = [&] {
        if (ahead.live) {
            uint4 *to = in + head * 128;
            const int64_t at = static_cast<int64_t>(ahead.h) * D + sub * 8;
            const uint16_t *x = a.x + ahead.t * a.x_stride + at, *g = a.dout + ahead.t * a.dout_stride + at;
            copy_async16(to, x);
            copy_async16(to + 32, x + HI);
            copy_async16(to + 64, g);
            copy_async16(to + 96, g + HI);
        }
        copy_commit();
        head = head + 1 == kBwdStages ? 0 : head + 1;
        ahead.next(a, first);
    };
    Positions pos;
    pos.load(a, now.t, now.live);
#pragma unroll 1
    for (int i = 0; i < kBwdStages - 1; ++i) copy();

    const uint16_t *w = (is_q ? a.wq : a.wk) + sub * 8;
    Pair wl[4], wh[4], dl[4], dh[4];  // weights; sums of g n^
    widen<E>(ld_ro16(w), wl);
    widen<E>(ld_ro16(w + HI), wh);
#pragma unroll
    for (int i = 0; i < 4; ++i) dl[i] = dh[i] = Pair::both(0.0f);

    while (now.inside()) {
        // R^T: the angles with the other sign, and no weights
        Turn<D, R, STYLE> back;
        const bool ok = pos.ok;
        if (now.live && !ok && sub == 0) atomicOr(&g_qk_axes_status, RN_STATUS_BAD_POSITION);
        {
            float c[8] = {}, s[8] = {};
            if (ok) lane_angles<D, R, STYLE>(a, pos, sub, c, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = -s[i];
            const Pair one[4] = {Pair::both(1.0f), Pair::both(1.0f), Pair::both(1.0f), Pair::both(1.0f)};
            back.set(c, s, one, one, one, sub);
        }
        {
            HeadPlace<L::TOKENS> then = now;  // the next unit's positions come meanwhile
            then.next_unit(a, first);
            pos.load(a, then.t, then.live);
        }
        bool end;
        do {
            copy_wait<kBwdStages - 2>();
            const uint4 *from = in + tail * 128;
            const uint4 ul = ld_shared16(from), uh = ld_shared16(from + 32);
            const uint4 vl = ld_shared16(from + 64), vh = ld_shared16(from + 96);
            tail = tail + 1 == kBwdStages ? 0 : tail + 1;
            copy();  // (to the stage that the head before came from)
            const float rstd = __frsqrt_rn(
                group_sum<L::LPH>(square_sum<E>(uh, square_sum<E>(ul, 0.0f))) / static_cast<float>(D) + a.eps);
            Pair x[4], y[4], p[4], q[4], o[4];
            widen<E>(vl, p);
            widen<E>(vh, q);
            widen<E>(partner<D, R, STYLE>(vl, sub), o);
            back.apply(p, q, o, sub);
            widen<E>(ul, x);
            widen<E>(uh, y);
            const Pair r = Pair::both(rstd);
            Pair dots = Pair::both(0.0f);
            // n^ = x rstd, dw += g n^, u = g w, dot = sum u n^
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = x[i] * r;
                y[i] = y[i] * r;
                if (ok) {
                    dl[i] = p[i].fma(x[i], dl[i]);
                    dh[i] = q[i].fma(y[i], dh[i]);
                }
                p[i] = p[i] * wl[i];
                q[i] = q[i] * wh[i];
                dots = p[i].fma(x[i], dots);
                dots = q[i].fma(y[i], dots);
            }
            const Pair dot = Pair::both(-group_sum<L::LPH>(dots.sum()) / static_cast<float>(D));
            if (ok) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[i] = r * x[i].fma(dot, p[i]);
                    q[i] = r * y[i].fma(dot, q[i]);
                }
                uint16_t *out = a.y + now.t * a.y_stride + static_cast<int64_t>(now.h) * D + sub * 8;
                st16(out, narrow<E>(p));
                st16(out + HI, narrow<E>(q));
            }
            end = now.next(a, first);
        } while (!end);
    }
    copy_wait<0>();
    __syncthreads();

    // the block's sums of dw, its groups in their order
    float *sums = reinterpret_cast<float *>(heads_in);
    float *mine = sums + (warp * L::TOKENS + lane / L::LPH) * D + sub * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<float2 *>(mine + 2 * i) = dl[i].v;
        *reinterpret_cast<float2 *>(mine + HI + 2 * i) = dh[i].v;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kBwdThreads) {
        float v = 0.0f;
#pragma unroll 8
        for (int g = 0; g < GROUPS; ++g) v += sums[g * D + d];
        a.partial[static_cast<int64_t>(blockIdx.x) * D + d] = v;
    }
}

// dw[which] (+)= the blocks' sums, in their order.  blockIdx.x: 32 dimensions, y: query or key.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) qk_axes_sum_kernel(const float *partial, int q_blocks, int blocks,
                                                                     int D, float *dwq, float *dwk, int accumulate) {
    __shared__ float sums[kSumWarps][33];
    pdl_trigger();
    float *dw = blockIdx.y == 0 ? dwq : dwk;
    if (!dw) return;
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b0 = blockIdx.y == 0 ? 0 : q_blocks, b1 = blockIdx.y == 0 ? q_blocks : blocks;
    float v = 0.0f;
#pragma unroll 8
    for (int b = b0 + warp; b < b1; b += kSumWarps) v += partial[static_cast<int64_t>(b) * D + blockIdx.x * 32 + lane];
    sums[warp][lane] = v;
    __syncthreads();
    v = warp_sum(sums[lane][warp]);  // dimension `warp` of the block's
    if (lane == 0) {
        const int d = blockIdx.x * 32 + warp;
        dw[d] = accumulate ? dw[d] + v : v;
    }
}

// ---- host -------------------------------------------------------------------------------


static int64_t bwd_workspace(int sm_count, int D) {
    return static_cast<int64_t>(sm_count) * kBwdBlocks * D * 4;
}

// Parts that `heads` heads are cut into so that a part has up to `most` of them.
static int parts_of(int heads, int most) { return (heads + most - 1) / most; }

// Heads of a part, at most: of 1, 2, 4 .. 32 what lets the last of `warps` warps end first, where
// to enter a unit costs a warp about as much as `enter` heads.
static int part_size(int64_t quads, int Hq, int Hkv, int64_t warps, int enter) {
    int best = 1;
    int64_t least = INT64_MAX;
    for (int n = 1; n <= 32; n *= 2) {
        const int64_t units = quads * (parts_of(Hq, n) + parts_of(Hkv, n));
        const int64_t cost = (units + warps - 1) / warps * (n + enter);
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

// A kernel with more than 48 KB of shared memory has to be told once on each device.
template <class Kernel>
static int allow_shared(Kernel kernel, int bytes, std::atomic<int> (&done)[kMaxDevices]) {
    const int idx = current_device_index();
    if (idx < 0 || idx >= kMaxDevices) return RN_ERR_DEVICE;
    if (done[idx].load(std::memory_order_acquire)) return RN_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return RN_ERR_DEVICE;
    }
    done[idx].store(1, std::memory_order_release);
    return RN_OK;
}

template <int D, int R, int STYLE, class E>
static int qk_axes_launch(QkAxesArgs &a, bool backward, float *dwq, float *dwk, int accumulate, const DeviceInfo &dev,
                          cudaStream_t st) {
    using L = AxesLane<D, R, STYLE>;
    static std::atomic<int> fwd_done[kMaxDevices], bwd_done[kMaxDevices];
    const int64_t quads = (a.T + L::TOKENS - 1) / L::TOKENS;
    // four pairs of one axis are one load of the table each way, of several eight
    int mixed = 0;
    for (int p = 0; p < R / 2; p += 4) {
        const uint32_t code = a.pair_axis[p >> 4] >> (2 * (p & 15)) & 0xFFu;
        if (code != (code & 3u) * 0x55u) mixed = 3;
    }
    const int n = backward ? part_size(quads, a.Hq, a.Hkv, static_cast<int64_t>(dev.sm_count) * kBwdBlocks * kBwdWarps,
                                       1 + mixed)
                           : part_size(quads, a.Hq, a.Hkv, static_cast<int64_t>(dev.sm_count) * kFwdBlocks * kFwdWarps,
                                       3 + mixed);
    a.part_heads = n;
    a.q_parts = parts_of(a.Hq, n);
    a.k_parts = parts_of(a.Hkv, n);
    const auto blocks_of = [&](int64_t units, int warps, int64_t cap) {
        const int64_t b = (units + warps - 1) / warps;
        return static_cast<int>(b < cap ? b : cap);
    };
    if (!backward) {
        constexpr int smem = kFwdWarps * kFwdStages * 1024;
        const int rc = allow_shared(qk_axes_fwd_kernel<D, R, STYLE, E>, smem, fwd_done);
        if (rc != RN_OK) return rc;
        const int blocks = blocks_of(quads * (a.q_parts + a.k_parts), kFwdWarps,
                                     static_cast<int64_t>(dev.sm_count) * kFwdBlocks);
        return launch_pdl(qk_axes_fwd_kernel<D, R, STYLE, E>, dim3(static_cast<unsigned>(blocks)), dim3(kFwdThreads),
                          smem, st, a);
    }
    constexpr int smem = kBwdWarps * kBwdStages * 2048;
    int rc = allow_shared(qk_axes_bwd_kernel<D, R, STYLE, E>, smem, bwd_done);
    if (rc != RN_OK) return rc;
    const int64_t most = static_cast<int64_t>(dev.sm_count) * kBwdBlocks;
    // shares of the grid by the heads, and the units that they are taken in
    const int64_t q_cost = a.Hq + a.q_parts, k_cost = a.Hkv + a.k_parts;
    int64_t q_cap = (most * q_cost + (q_cost + k_cost) / 2) / (q_cost + k_cost);
    if (q_cap < 1) q_cap = 1;
    if (q_cap > most - 1) q_cap = most - 1;
    a.q_blocks = blocks_of(quads * a.q_parts, kBwdWarps, a.Hkv ? q_cap : most);
    const int k_blocks = blocks_of(quads * a.k_parts, kBwdWarps, a.Hq ? most - q_cap : most);
    const int blocks = a.q_blocks + k_blocks;
    rc = launch_pdl(qk_axes_bwd_kernel<D, R, STYLE, E>, dim3(static_cast<unsigned>(blocks)), dim3(kBwdThreads), smem,
                    st, a);
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
    if (H > INT32_MAX - 64 || (H > 0 && a.T > INT32_MAX / H)) return RN_ERR_SHAPE;
    if (a.max_pos < 1 || a.max_pos > INT32_MAX) return RN_ERR_SHAPE;
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
    // in place is row by row
    if (a.T > 1 && !empty &&
        ((a.y == a.x && a.y_stride != a.x_stride) || (k.backward && a.y == a.dout && a.y_stride != a.dout_stride)))
        return RN_ERR_ARG;
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
