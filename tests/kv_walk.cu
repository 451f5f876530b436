// kv_walk.cu -- runs the walk of the attention kernels' CTAs over their work on the
// host: every piece that the joining kernel follows has to be noted, also by a CTA whose
// waits ran out, and the notes have to say where the pieces are.  Prints the number of
// layouts looked at; the first fault ends it with status 1.
#include <stdio.h>

#include <random>
#include <vector>

#include "../row_normalization_gb300/csrc/kv_attention.cuh"

using namespace rn;

static int g_cut_heads = 0;

#define REQUIRE(x)                                                \
    do {                                                          \
        if (!(x)) {                                               \
            printf("line %d: %s (layout %d)\n", __LINE__, #x, n); \
            return 1;                                             \
        }                                                         \
    } while (0)

// One layout: the call of `lens` and `nq` laid on `grid` CTAs, whose threads give up in
// front of their run number `give_up` (large: never).
template <class L, int SLOT>
static int check_layout(int n, const std::vector<int32_t> &lens, const std::vector<int64_t> &nq, int hkv, int group,
                        int grid, int window, int sinks, int give_up) {
    std::vector<int64_t> cu(1, 0);
    int64_t most = 1;
    for (int64_t x : nq) {
        cu.push_back(cu.back() + x);
        if (x > most) most = x;
    }
    KvAttnArgs a = {};
    a.cache.Hkv = hkv;
    a.cache.log2_page = 4;
    a.B = static_cast<int64_t>(lens.size());
    a.max_pages = 1 << 20;
    a.kv_lens = lens.data();
    a.cu_q = cu.data();
    a.T = cu.back();
    a.max_q_len = most;
    a.most_q = INT64_MAX;
    a.group = group;
    a.Hq = group * hkv;
    a.window = window;
    a.sinks = sinks;
    a.q_tiles = (most * group + L::NQ - 1) / L::NQ;
    a.heads = a.B * a.q_tiles * hkv;
    a.grid = grid;
    std::vector<CutNote> notes(grid);
    for (CutNote &x : notes) x.row0 = x.f0 = x.ncols = x.head0 = x.pieces = x.first_slot = -77;
    a.cuts = notes.data();
    a.partial = reinterpret_cast<float *>(1 << 20);  // (only its differences are looked at)

    int64_t line = 0;
    const int64_t items = a.B * a.q_tiles;
    for (int64_t i = 0; i < items; ++i) line += make_item<L>(a, i).units();
    if (line == 0) return 0;
    const Cut<L> cut(line * hkv, grid);
    REQUIRE(cut.start(cut.ctas) == line * hkv);
    struct Piece {
        int64_t slot;
        int k0, k1;
    };
    std::vector<std::vector<Piece>> pieces(items * hkv);
    for (int64_t cta = 0; cta < cut.ctas; ++cta) {
        int64_t item = 0, before = 0;
        for (;; ++item) {
            const int64_t units = make_item<L>(a, item).units();
            if (cut.start(cta) < (before + units) * hkv) break;
            before += units;
        }
        // a thread whose waits hold: all runs of the CTA, as (item, head) by its first column
        walk_runs<SLOT>(a, cut, cta, item, before, 0, false,
                        [&](const Item<L> &it, int head, int k0, int k1, float *part) {
                            const int64_t i = it.seq * a.q_tiles + it.f0 / L::NQ;
                            pieces[i * hkv + head].push_back({part ? (part - a.partial) / SLOT : -1, k0, k1});
                            return true;
                        });
        // one that gives up ends there
        int calls = 0;
        const auto body = [&](const Item<L> &, int, int, int, float *) { return calls++ != give_up; };
        walk_runs<SLOT>(a, cut, cta, item, before, 0, false, body);
        REQUIRE(calls <= give_up + 1);
        // but the one that notes
        calls = 0;
        walk_runs<SLOT>(a, cut, cta, item, before, 0, true, body);
        REQUIRE(calls <= give_up + 1);
    }
    const bool by_head = a.heads <= grid;
    std::vector<bool> found(items * hkv, false);
    for (int64_t i = 0; i < (by_head ? a.heads : cut.ctas); ++i) {
        const CutNote &x = notes[i];
        if (by_head && make_item<L>(a, i / hkv).n == 0) continue;  // the kernel clears these apart
        REQUIRE(x.pieces == 0 || x.pieces >= 2);
        if (x.pieces == 0) continue;
        int64_t i0 = -1;  // whose it is
        for (int64_t k = 0; k < items; ++k) {
            const Item<L> it = make_item<L>(a, k);
            if (it.n > 0 && it.row0 == x.row0 && it.f0 == x.f0 && it.ncols == x.ncols) i0 = k;
        }
        REQUIRE(i0 >= 0 && x.head0 % group == 0 && x.head0 / group < hkv);
        const int64_t at = i0 * hkv + x.head0 / group;
        REQUIRE(!by_head || at == i);
        REQUIRE(!found[at]);
        found[at] = true;
        const auto &ps = pieces[at];
        REQUIRE(static_cast<int>(ps.size()) == x.pieces);
        for (int p = 0; p < x.pieces; ++p)
            REQUIRE(ps[p].slot == (p == 0 ? x.first_slot : (x.first_slot & ~1) + 2 * p) && ps[p].slot < 2 * grid);
    }
    for (int64_t i = 0; i < items * hkv; ++i) {
        const Item<L> it = make_item<L>(a, i / hkv);
        int at = 0;
        for (const Piece &p : pieces[i]) {
            REQUIRE(p.k0 == at && p.k1 > p.k0);
            at = p.k1;
            REQUIRE((p.slot < 0) == (pieces[i].size() == 1));
        }
        REQUIRE(at == it.n && found[i] == (pieces[i].size() > 1));
        g_cut_heads += found[i];
    }
    return 0;
}

int main() {
    using Narrow = LineShape<8, 32, 16, 4>;
    using Wide = LineShape<256, 128, 4, 1>;
    std::mt19937 rng(1);
    const auto pick = [&](int lo, int hi) { return lo + static_cast<int>(rng() % (hi - lo + 1)); };
    int n = 0;
    for (; n < 3000; ++n) {
        const int B = pick(1, 20), hkv = pick(1, 5), group = pick(1, 8), grid = pick(1, 60);
        const int window = pick(0, 3) ? 0 : pick(1, 700), sinks = pick(0, 40), give_up = pick(0, 5) ? pick(0, 6) : 1 << 30;
        std::vector<int32_t> lens;
        std::vector<int64_t> nq;
        for (int b = 0; b < B; ++b) {
            lens.push_back(pick(0, 2) ? pick(0, 9000) : pick(0, 40));
            nq.push_back(pick(0, 4) ? 1 : pick(0, 300));
        }
        const int rc = n & 1 ? check_layout<Wide, 100>(n, lens, nq, hkv, group, grid, window, sinks, give_up)
                             : check_layout<Narrow, 100>(n, lens, nq, hkv, group, grid, window, sinks, give_up);
        if (rc) return rc;
    }
    printf("%d layouts, %d cut heads\n", n, g_cut_heads);
    return 0;
}
