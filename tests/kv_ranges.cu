// Host check of how attention's work is cut up: walks every block's range of random batches as the kernels do and compares with the
// units counted one by one.  Prints "ok <cases> <largest total>" or the first difference.
#include <stdio.h>
#include <stdlib.h>

#include <map>
#include <random>
#include <vector>

#include "sv_attend.cuh"

using namespace sv;

static std::mt19937_64 rng(1);
static long long upto(long long n) { return (long long)(rng() % (unsigned long long)(n + 1)); }

#define CHECK(x, ...)                                      \
    do {                                                   \
        if (!(x)) {                                        \
            printf("line %d: %s ", __LINE__, #x);          \
            printf(__VA_ARGS__);                           \
            printf("\n");                                  \
            exit(1);                                       \
        }                                                  \
    } while (0)

struct Part {
    int block, k0, k1;
    size_t slot;
};

// One launch over segments [s0, s1) of a: returns its total.
static long long check_launch(AttendArgs a, const AttendTiles &tiles, int s0, int s1, int blocks, size_t slot0, size_t slots) {
    AttendGeo &geo = a.geo;
    geo.s0 = s0;
    geo.s1 = s1;
    geo.blocks = blocks;
    geo.slot0 = slot0;
    geo.set(tiles);
    std::vector<long long> off(s1 - s0 + 1);
    std::vector<int> per(s1 - s0);
    geo.seg_off = off.data();
    long long total = 0;
    for (int s = s0; s < s1; ++s) {
        const Seg g = seg_of(a, geo, s, false);
        off[s - s0] = total;
        per[s - s0] = units_before(a, geo, g, g.tiles_m);
        CHECK(per[s - s0] >= 0, "segment %d", s);
        total += (long long)per[s - s0] * a.c.kv_heads;
    }
    off[s1 - s0] = total;
    const Ranges r = ranges_of(total, geo);
    CHECK(total == 0 || (r.parts >= 1 && r.parts <= blocks && range_start(r, r.parts) == total), "total %lld", total);

    std::map<std::pair<int, std::pair<int, int>>, std::vector<Part>> parts;   // (segment, key head, row tile) -> pieces
    std::vector<AttendTail> tails(blocks);
    for (int c = 0; c < blocks; ++c) {
        Walk w{};
        w.total = total;
        const long long pos = c < r.parts ? range_start(r, c) : total;
        w.stop = c < r.parts ? range_start(r, c + 1) : total;
        CHECK(c >= r.parts || w.stop - pos == r.each + (c < r.more), "block %d", c);
        w.head_at = w.stop;
        for (int s = s0; s < s1 && pos < w.stop; ++s)
            if (pos >= off[s - s0] && pos < off[s - s0 + 1]) w.begin(seg_of(a, geo, s, false), s, per[s - s0], off[s - s0], pos);
        Piece p;
        for (bool first = true, more = true; more; first = false) {
            more = w.next(a, p);
            if (first) tails[c] = tail_of(a, w, p, more);
            if (!more) break;
            CHECK(p.k0 >= 0 && p.k0 < p.k1 && p.k1 <= p.kt && p.vr > 0 && p.vr <= geo.TM, "block %d", c);
            const size_t slot = unit_slot(a, geo, p.g, p.seg < a.n_groups, p.h, p.t) + (size_t)c * geo.TM;
            CHECK(slot >= slot0 && slot + p.vr <= slots, "slot %zu of %zu", slot, slots);
            parts[{p.seg, {p.h, p.t}}].push_back({c, p.k0, p.k1, slot});
        }
    }
    std::map<size_t, size_t> used;   // slots [first, end)
    size_t units = 0, n_tails = 0;
    for (int s = s0; s < s1; ++s) {
        const Seg g = seg_of(a, geo, s, false);
        for (int h = 0; h < a.c.kv_heads; ++h) {
            const JoinSeg js = join_seg(a, geo, s, h);
            for (int t = 0; t < g.tiles_m; ++t) {
                const int kt = seg_tiles(a, geo, g, t), vr = std::min(geo.TM, g.packed - t * geo.TM);
                const auto &v = parts[{s, {h, t}}];
                const JoinUnit u = join_unit(a, geo, js, t);
                if (kt <= 0) {
                    CHECK(v.empty() && u.c1 < u.c0, "empty unit");
                    continue;
                }
                ++units;
                int at = 0;
                for (const Part &q : v) {
                    CHECK(q.k0 == at, "segment %d head %d rows %d: tile %d after %d", s, h, t, q.k0, at);
                    at = q.k1;
                    auto it = used.upper_bound(q.slot);
                    CHECK((it == used.end() || it->first >= q.slot + vr) && (it == used.begin() || (--it)->second <= q.slot), "slots shared");
                    used[q.slot] = q.slot + vr;
                }
                CHECK(at == kt, "segment %d head %d rows %d: %d of %d tiles", s, h, t, at, kt);
                CHECK(u.c0 == v.front().block && u.c1 == v.back().block && u.tiles == kt, "join's blocks");
                size_t i = 0;
                for (int c = u.c0; c <= u.c1; ++c) {
                    const bool has = i < v.size() && v[i].block == c;
                    CHECK(has == block_has(js.r, c, u.at, u.cost, u.tiles), "block %d of a unit", c);
                    i += has;
                }
                CHECK(i == v.size(), "pieces");
                if (v.size() > 1) {   // its tail
                    const AttendTail &q = tails[v.back().block];
                    CHECK(block_of_place(ranges_of(q.total, geo), q.at) == u.c0 && q.at == u.at && q.total == total && q.tiles == kt, "tail");
                    CHECK(q.r0 == g.r0 && q.m0 == t * geo.TM && q.vr == vr && q.h == h, "tail's rows");
                    for (const Part &x : v) CHECK((size_t)q.slot + (size_t)x.block * geo.TM == x.slot, "tail's slots");
                    ++n_tails;
                }
            }
        }
    }
    for (const AttendTail &q : tails) n_tails -= q.tiles > 0;
    CHECK(n_tails == 0, "tails of nothing");
    for (auto &v : parts) units -= !v.second.empty();
    CHECK(units == 0, "pieces of nothing");
    return total;
}

int main(int argc, char **argv) {
    const int cases = argc > 1 ? atoi(argv[1]) : 300;
    long long largest = 0;
    for (int k = 0; k < cases; ++k) {
        const bool huge = k % 3 == 2, ragged = upto(2) == 0, tree = !ragged && upto(2) == 0, groups = upto(1);
        AttendArgs a{};
        KvBatch &bt = a.bt;
        bt.B = 1 + (int)upto(huge ? 60 : 40);
        bt.n = 1 + (int)upto(tree ? 128 : huge ? 3000 : 200);
        a.c.kv_heads = 1 + (int)upto(6);
        a.G = 1 << upto(3);
        a.q_heads = a.G * a.c.kv_heads;
        a.c.page_size = 1 << upto(16);
        const long long slots = huge ? 2147483647LL - 1024 : 20000;
        bt.max_pages = std::max(1, (int)(slots / a.c.page_size));
        const long long cap = (long long)bt.max_pages * a.c.page_size;
        std::vector<int> starts(bt.B + 1), ctx(bt.B), gs, pre;
        for (int b = 0; b < bt.B; ++b) starts[b + 1] = starts[b] + (ragged ? (int)upto(bt.n) : bt.n);
        bt.rows = starts[bt.B];
        if (ragged) bt.row_start = starts.data();
        static int parents[1];
        if (tree) bt.parents = parents;   // only looked at for being there
        for (int &c : ctx) c = (int)std::min(cap - bt.n, huge ? (long long)upto(cap) : (1LL << upto(14)) - 1 + upto(300));
        if (groups) {
            for (int b = 0; b < bt.B; b += 1 + (int)upto(8)) gs.push_back(b);
            gs.push_back(bt.B);
            for (size_t g = 0; g + 1 < gs.size(); ++g) {
                int low = ctx[gs[g]];
                for (int b = gs[g]; b < gs[g + 1]; ++b) low = std::min(low, ctx[b]);
                pre.push_back((int)upto(low));
            }
            a.n_groups = (int)pre.size();
            a.group_start = gs.data();
            a.prefix_len = pre.data();
        }
        bt.context_len = ctx.data();
        const int blocks = 1 + (int)upto(319), n_seg = a.n_groups + bt.B;
        const int64_t own = (int64_t)bt.n * a.G, all = (int64_t)bt.rows * a.G;
        for (const AttendTiles &t : {kTilesTall, tiles_f32(64, 128), tiles_f32(64, 256)}) {
            if (!tiles_fit(t, groups ? std::max(own, all) : own, cap)) continue;
            largest = std::max(largest, check_launch(a, t, 0, n_seg, blocks, 0, attend_slots(bt.rows, a.q_heads, groups, true, t.TM, blocks)));
        }
        for (const AttendTiles &t : {kTilesFew, tiles_few32(4), tiles_few32(8), tiles_f32(16, 256)}) {
            if (own > t.TM) continue;
            const size_t slot0 = groups ? attend_slots(bt.rows, a.q_heads, true, false, 256, blocks) : 0;
            largest = std::max(largest, check_launch(a, t, a.n_groups, n_seg, blocks, slot0,
                                                     slot0 + attend_slots(bt.rows, a.q_heads, false, true, t.TM, blocks)));
        }
    }
    printf("ok %d %lld\n", cases, largest);
    return 0;
}
