// kv_attention.cuh -- what the two attention kernels over the quantised cache
// share: the call's arguments, the line of work units and its cut into runs, the
// store of a finished column and the joining of pieces.
#pragma once

#include "kv_common.cuh"

namespace rn {

// Each translation unit's own status word; rn_device_status() ORs them.
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
    int64_t min_q, most_q;  // sequences with fewer or more queries are another launch's
    int Hq;
    int group;         // query heads of a kv head
    float scale_log2;  // softmax scale * log2(e)
    int window;        // 0: none
    int sinks;
    uint16_t *out;
    float *lse;
    // workspace: the line's length, what each CTA's start cuts [grid], the partial sums
    int64_t *units;
    struct CutNote *cuts;
    float *partial;
    int64_t q_tiles;   // query tiles of a sequence
    int64_t heads;     // (query tile, kv head)s in all
    int grid;          // CTAs of the attention kernel
    bool direct;       // one for each (query tile, kv head) instead
};

// A (query tile, head) cut into pieces, with all the joining kernel needs of it; noted
// by the CTA of its second piece, so once.  The notes are one for each (query tile,
// head) where these are fewer than the CTAs, else one for each CTA; pieces 0: none.
struct CutNote {
    int64_t row0;       // as Item
    int32_t f0, ncols;
    int32_t head0;      // first query head
    int32_t pieces;
    int32_t first_slot; // of the first piece; the others lie two on from an even slot each
    int32_t unused;
};

// How a kernel lays its work on the line: NQ columns (queries of the tile times
// heads of the group) by tiles of TILE tokens, LEAD units without work in front of
// each (query tile, head) for what it costs to begin and end one, and runs of
// MIN units or more.
template <int NQ_, int TILE_, int LEAD_, int MIN_>
struct LineShape {
    static constexpr int NQ = NQ_, TILE = TILE_, LEAD = LEAD_, MIN = MIN_;
};

// 2^x to 2^-22 of it, and zero below 2^-126: the weights are rounded to 2^-11 behind it,
// and the factors that join sums are as good as the sums.
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One (sequence, query tile): its columns and the tiles of tokens they see.
template <class L>
struct Item {
    int64_t seq;     // the sequence
    int64_t row0;    // its first query row
    int f0, ncols;   // columns f0 .. f0 + ncols - 1 of the sequence's n_q * group
    int pos0;        // position of the sequence's first query
    int lo_pos, hi;  // position of the first column's query; one past the last column's
    int win_lo;      // first token inside the first column's window (0 without one)
    int sink_tiles;  // tiles 0 .. sink_tiles - 1, then lo_tile ..
    int lo_tile;
    int n;           // tiles in all
    bool bad;        // something had to be cut to the tensors

    // its units on the line, for one head
    __host__ __device__ __forceinline__ int units() const { return n > 0 ? n + L::LEAD : 0; }

    __host__ __device__ __forceinline__ int token(int k) const {
        return (k < sink_tiles ? k : lo_tile + (k - sink_tiles)) * L::TILE;
    }
};

template <class L>
__host__ __device__ __forceinline__ Item<L> make_item(const KvAttnArgs &a, int64_t item) {
    Item<L> it;
    uint32_t b = static_cast<uint32_t>(item), qt = 0;  // items fit 31 bits
    if (a.q_tiles != 1) {
        b = static_cast<uint32_t>(item) / static_cast<uint32_t>(a.q_tiles);
        qt = static_cast<uint32_t>(item) - b * static_cast<uint32_t>(a.q_tiles);
    }
    it.seq = b;
    it.bad = false;
    int64_t nq = 1;
    it.row0 = b;
    if (a.cu_q) {
        it.row0 = a.cu_q[b];
        const int64_t end = a.cu_q[b + 1];
        it.bad = end > it.row0 && (it.row0 < 0 || end > a.T);
        nq = end > it.row0 && !it.bad ? end - it.row0 : 0;  // (no difference of wild numbers)
        if (nq < a.min_q || nq > a.most_q) nq = 0;
    }
    int64_t len = a.kv_lens[b];
    const int64_t room = a.max_pages << a.cache.log2_page;
    if (len > room) {
        it.bad = true;
        len = room;
    }
    if (len < 0) len = 0;
    it.pos0 = static_cast<int>(len - nq);
    if (nq > a.max_q_len) {
        it.bad = true;
        nq = a.max_q_len;
    }
    const int64_t left = nq * a.group - static_cast<int64_t>(qt) * L::NQ;
    it.f0 = static_cast<int>(qt * L::NQ);
    it.ncols = static_cast<int>(left < 0 ? 0 : (left < L::NQ ? left : L::NQ));
    it.lo_pos = it.pos0 + it.f0 / a.group;
    it.hi = it.pos0 + (it.f0 + it.ncols - 1) / a.group + 1;
    it.win_lo = it.sink_tiles = it.lo_tile = it.n = 0;
    if (it.ncols == 0 || it.hi <= 0) return it;
    const int tiles = (it.hi + L::TILE - 1) / L::TILE;
    if (a.window && it.lo_pos >= a.window) {
        it.win_lo = it.lo_pos - a.window + 1;
        it.sink_tiles = a.sinks >= it.hi ? tiles : (a.sinks + L::TILE - 1) / L::TILE;
        if (it.sink_tiles > tiles) it.sink_tiles = tiles;
        it.lo_tile = it.win_lo / L::TILE;
        if (it.lo_tile < it.sink_tiles) it.lo_tile = it.sink_tiles;
    }
    it.n = it.sink_tiles + tiles - it.lo_tile;
    return it;
}

// a / b, in 32 bits where both fit (they nearly always do).
__host__ __device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The line cut into runs for its CTAs, the first `rest` of them one unit longer.
template <class L>
struct Cut {
    int64_t ctas, run, rest;

    __host__ __device__ __forceinline__ Cut(int64_t units, int grid) {
        const int64_t want = (units + L::MIN - 1) / L::MIN;
        ctas = want < grid ? (want > 0 ? want : 1) : grid;
        run = quotient(units, ctas);
        rest = units - run * ctas;
    }
    __host__ __device__ __forceinline__ int64_t start(int64_t c) const { return c * run + (c < rest ? c : rest); }
    __host__ __device__ __forceinline__ int64_t cta_of(int64_t unit) const {
        const int64_t longer = rest * (run + 1);
        return unit < longer ? quotient(unit, run + 1) : rest + quotient(unit - longer, run);
    }
};

// Four dimensions of a finished column: out = sum / l (the codes' 2^-24 undone),
// lse = (reference + log2(l)) ln 2.
template <int D, class L>
__device__ __forceinline__ void store_result(const KvAttnArgs &a, const Item<L> &it, int head0, int col, int d0,
                                             float4 v, float ref, float l) {
    const int f = it.f0 + col;
    const int64_t t = it.row0 + f / a.group;
    const int64_t row = t * a.Hq + head0 + f % a.group;
    const float inv = l == 0.0f ? 0.0f : 0x1p24f / l;
    const uint2 w = make_uint2(pack_bf2(v.x * inv, v.y * inv), pack_bf2(v.z * inv, v.w * inv));
    *reinterpret_cast<uint2 *>(a.out + row * D + d0) = w;
    if (d0 == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
}

// Sum of the item sizes before this thread's share, by a scan over the block;
// every CTA runs it over all items, so that no launch has to come before.
struct Line {
    int64_t units;        // in all, over every kv head
    int64_t item, before; // the item at a wanted unit, and the units of one head before it
};

template <class L, int THREADS>
__device__ __forceinline__ Line find_unit(const KvAttnArgs &a, bool publish, int64_t *scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t items = a.B * a.q_tiles;
    const int64_t per = (items + THREADS - 1) / THREADS;
    const int64_t i0 = tid * per < items ? tid * per : items;
    const int64_t i1 = i0 + per < items ? i0 + per : items;
    int64_t sum = 0;
    bool bad = false;
    for (int64_t i = i0; i < i1; ++i) {
        const Item<L> it = make_item<L>(a, i);
        sum += it.units();
        bad |= it.bad;
    }
    if (publish && bad) atomicOr(&g_kv_attention_status, RN_STATUS_BAD_INDEX);
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    Line line;
    line.units = total * a.cache.Hkv;
    if (publish && tid == 0) *a.units = line.units;
    const Cut<L> cut(line.units, a.grid);
    const int64_t u = cut.start(blockIdx.x);
    if (blockIdx.x < cut.ctas && before * a.cache.Hkv <= u && u < (before + sum) * a.cache.Hkv) {
        int64_t run = before, i = i0;
        for (; i + 1 < i1; ++i) {
            const int n = make_item<L>(a, i).units();
            if (u < (run + n) * a.cache.Hkv) break;
            run += n;
        }
        scratch[THREADS / 32] = i;
        scratch[THREADS / 32 + 1] = run;
    }
    __syncthreads();
    line.item = scratch[THREADS / 32];
    line.before = scratch[THREADS / 32 + 1];
    return line;
}

// Zeros for the rows of an item that sees no token, of one kv head.
template <int D, class L, int THREADS>
__device__ __forceinline__ void store_zeros(const KvAttnArgs &a, const Item<L> &it, int head) {
    for (int idx = threadIdx.x; idx < it.ncols * (D / 4); idx += THREADS)
        store_result<D>(a, it, head * a.group, idx / (D / 4), idx % (D / 4) * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f),
                        0.0f, 0.0f);
}

// The same of every such item, shared out over the CTAs.
template <int D, class L, int THREADS>
__device__ __forceinline__ void store_empty(const KvAttnArgs &a) {
    const int64_t items = a.B * a.q_tiles;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const Item<L> it = make_item<L>(a, i);
        if (it.n > 0) continue;
        if (a.heads <= a.grid)
            for (int h = threadIdx.x; h < a.cache.Hkv; h += THREADS) a.cuts[i * a.cache.Hkv + h].pieces = 0;
        for (int head = 0; head < a.cache.Hkv; ++head) store_zeros<D, L, THREADS>(a, it, head);
    }
}

// Notes for the joining kernel on the piece [v0, v1) of `units` units of a (query
// tile, head) whose first unit is `first`; by one thread of CTA `cta`.
template <class L>
__host__ __device__ __forceinline__ void note_piece(const KvAttnArgs &a, const Cut<L> &cut, int64_t cta, int64_t first,
                                                    int v0, int v1, int units, const Item<L> &it, int64_t item,
                                                    int head) {
    const int64_t c0 = cta - 1;
    // the second piece: the CTA before holds the first unit with work
    const bool second = v0 > L::LEAD && cut.start(c0) <= first + L::LEAD;
    const bool by_head = a.heads <= a.grid;
    const bool none = by_head ? v0 <= L::LEAD && v1 == units : !second && first + v0 == cut.start(cta);
    if (!second && !none) return;
    CutNote n;
    n.row0 = it.row0;
    n.f0 = it.f0;
    n.ncols = it.ncols;
    n.head0 = head * a.group;
    n.pieces = second ? static_cast<int>(cut.cta_of(first + units - 1) - c0) + 1 : 0;
    n.first_slot = static_cast<int>(2 * c0 + (cut.start(c0) < first ? 1 : 0));
    n.unused = 0;
    a.cuts[by_head ? item * a.cache.Hkv + head : cta] = n;
}

// Calls body(item, head, first tile, end, slot for a piece or null) for each run of CTA
// `cta` of the line, which begins at `item` with `before` units of one head in front of
// it, or for its only (query tile, head) where a.direct.  A body that returns false (its
// wait ran out) is the thread's last; but the thread that notes walks on and notes every
// piece, for the joining kernel follows the notes whatever became of the sums.
#pragma nv_exec_check_disable
template <int SLOT, class L, class Body>
__host__ __device__ __forceinline__ void walk_runs(const KvAttnArgs &a, const Cut<L> &cut, int64_t cta, int64_t item,
                                                   int64_t before, int own_head, bool notes, Body &&body) {
    const int64_t u0 = a.direct ? 0 : cut.start(cta), u1 = a.direct ? 1 : cut.start(cta + 1);
    int64_t u = u0;
    bool ok = true;
    while (u < u1) {
        const Item<L> it = make_item<L>(a, item);
        if (it.n == 0) {
            ++item;
            continue;
        }
        int units = 1, head = own_head, v0 = 0, v1 = 1, k0 = 0, k1 = it.n;
        if (!a.direct) {
            units = it.units();
            const int64_t in = u - before * a.cache.Hkv;
            head = static_cast<int>(quotient(in, units));
            v0 = static_cast<int>(in - static_cast<int64_t>(head) * units);
            const int64_t left = u1 - u;
            v1 = units - v0 <= left ? units : v0 + static_cast<int>(left);
            k0 = v0 > L::LEAD ? v0 - L::LEAD : 0;
            k1 = v1 - L::LEAD;
        }
        if (ok && k1 > k0) {
            float *part = nullptr;
            if (k1 - k0 != it.n) part = a.partial + (2 * cta + (u == u0 ? 0 : 1)) * SLOT;
            ok = body(it, head, k0, k1, part);
        }
        if (!a.direct && notes) note_piece(a, cut, cta, u - v0, v0, v1, units, it, item, head);
        if (!ok && !notes) return;
        u += v1 - v0;
        if (v1 == units && head == a.cache.Hkv - 1) {
            before += units;
            ++item;
        }
    }
}

constexpr int kJoinWarps = 8;
constexpr int64_t kJoinBlocks = 2432;  // about sixteen an SM
constexpr int kEarly = 4;      // pieces a warp loads ahead
constexpr int kFewPieces = 8;  // pieces that one warp joins by itself

// ---- joining the pieces of a cut (query tile, head) -------------------------------------

// blockIdx.x: a note on a cut (query tile, head), y: a share of the columns' quads of
// dimensions.  A lane owns four dimensions of a column; a warp takes all pieces of its
// columns where they are few, else the warps share them.
template <int D, class L>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_attention_join_kernel(const KvAttnArgs a) {
    constexpr int NQ = L::NQ, SLOT = NQ * (D + 2), QUADS = D / 4;
    constexpr int W = QUADS < 32 ? QUADS : 32;  // lanes of one column
    __shared__ float4 s_acc[kJoinWarps][32];
    __shared__ float s_ref[kJoinWarps][32], s_l[kJoinWarps][32];
    pdl_trigger();
    pdl_wait();
    const int64_t units = *a.units;
    const CutNote note = a.cuts[blockIdx.x];
    if (units == 0 || (a.heads > a.grid && blockIdx.x >= Cut<L>(units, a.grid).ctas)) return;
    const int pieces = note.pieces;
    if (pieces == 0) return;
    Item<L> it;
    it.row0 = note.row0;
    it.f0 = note.f0;
    it.ncols = note.ncols;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // all pieces but the first are the first of their CTAs
    const float *first_part = a.partial + static_cast<int64_t>(note.first_slot) * SLOT;
    const float *parts = a.partial + static_cast<int64_t>(note.first_slot & ~1) * SLOT;
    const auto piece = [&](int p) { return p == 0 ? first_part : parts + static_cast<int64_t>(p) * 2 * SLOT; };
    const bool share = pieces > kFewPieces;
    const int p0 = share ? warp : 0, step = share ? kJoinWarps : 1;
    const int chunk0 = share ? blockIdx.y : blockIdx.y * kJoinWarps + warp;
    const int chunks = share ? gridDim.y : gridDim.y * kJoinWarps;
    for (int base = chunk0 * 32; base < it.ncols * QUADS; base += 32 * chunks) {
        const int col = (base + lane) / QUADS, d0 = (base + lane) % QUADS * 4;
        const bool live = col < it.ncols;
        // the largest reference of the warp's pieces and their sum of weights, by the
        // column's lanes together
        float top = -INFINITY, l = 0.0f;
        // (the first pieces' sums come while their references are looked at)
        float4 early[kEarly];
        if (live)
#pragma unroll
            for (int i = 0; i < kEarly; ++i)
                if (p0 + i * step < pieces)
                    early[i] = *reinterpret_cast<const float4 *>(piece(p0 + i * step) + col * D + d0);
        if (live)
            for (int p = p0 + step * (lane % W); p < pieces; p += step * W) top = fmaxf(top, piece(p)[NQ * D + col]);
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float ref = top == -INFINITY ? 0.0f : top;
        if (live)
            for (int p = p0 + step * (lane % W); p < pieces; p += step * W)
                l = fmaf(piece(p)[NQ * D + NQ + col], exp2_approx(piece(p)[NQ * D + col] - ref), l);
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const auto add = [&](const float *part, float4 v) {
            const float f = exp2_approx(part[NQ * D + col] - ref);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        };
        if (live) {
#pragma unroll
            for (int i = 0; i < kEarly; ++i)
                if (p0 + i * step < pieces) add(piece(p0 + i * step), early[i]);
#pragma unroll 8
            for (int p = p0 + kEarly * step; p < pieces; p += step)
                add(piece(p), *reinterpret_cast<const float4 *>(piece(p) + col * D + d0));
        }
        if (share) {
            s_acc[warp][lane] = acc;
            s_ref[warp][lane] = top;
            s_l[warp][lane] = l;
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, s_ref[w][lane]);
                ref = top == -INFINITY ? 0.0f : top;
                acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                l = 0.0f;
                for (int w = 0; w < kJoinWarps; ++w) {
                    const float f = exp2_approx(s_ref[w][lane] - ref);
                    const float4 v = s_acc[w][lane];
                    l = fmaf(s_l[w][lane], f, l);
                    acc.x = fmaf(v.x, f, acc.x);
                    acc.y = fmaf(v.y, f, acc.y);
                    acc.z = fmaf(v.z, f, acc.z);
                    acc.w = fmaf(v.w, f, acc.w);
                }
            }
            __syncthreads();
        }
        if (live && (!share || warp == 0)) store_result<D, L>(a, it, note.head0, col, d0, acc, ref, l);
    }
}

// Launches the joining kernel behind an attention kernel on the same stream.
template <int D, class L>
static int join_launch(const KvAttnArgs &a, cudaStream_t st) {
    // blocks for the GPU to be full of them, as far as there is work for a warp (few
    // pieces) or a block (many) in each
    constexpr int64_t kChunks = L::NQ * D / 4 / 32;
    const int64_t notes = a.heads < a.grid ? a.heads : a.grid;
    const int64_t most = a.grid > kFewPieces * a.heads ? kChunks : (kChunks + kJoinWarps - 1) / kJoinWarps;
    int64_t shares = (kJoinBlocks + notes - 1) / notes;
    if (shares > most) shares = most;
    return launch_pdl(kv_attention_join_kernel<D, L>, dim3(static_cast<unsigned>(notes), static_cast<unsigned>(shares)),
                      dim3(32 * kJoinWarps), 0, st, a);
}

// ---- host: how a call is laid out ------------------------------------------------------------

struct AttnPlan {
    int64_t q_tiles;
    int grid;
    int64_t head_bytes;  // of the workspace, before the partial sums
    int64_t bytes;
};

// The most tokens a query tile of `columns` can see: the table's, or the window's (and
// the ends of tiles) and the sinks'.
inline int64_t attn_most_tokens(const KvAttnArgs &a, int columns) {
    const int64_t room = a.max_pages << a.cache.log2_page;
    if (!a.window) return room;
    const int64_t few = static_cast<int64_t>(a.window) + columns / a.group + 64 + (a.sinks < room ? a.sinks : room);
    return few < room ? few : room;
}

// About how many (query tile, kv head)s have work: by the queries there are, not those that
// max_q_len allows for.  (The second launch of a mixed call counts on few sequences: of 16
// one with 60 queries over 2000 tokens took 50 us with a CTA for each head, 32 on the line,
// when this was chosen.)
inline int64_t attn_busy_heads(const KvAttnArgs &a, int columns) {
    const int64_t busy = (a.T * a.group / columns + (a.min_q > 1 ? 1 : a.B)) * a.cache.Hkv;
    return busy < a.heads ? busy : a.heads;
}

// kv_attention_wide.cu: 128 columns at a time.
AttnPlan wide_plan(int sm_count, int64_t B, int group, int D, int64_t max_q_len);
int wide_launch(int D, int format, KvAttnArgs &a, cudaStream_t st);

}  // namespace rn
