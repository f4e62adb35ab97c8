// sv_attend.cuh — how sv_kv_attend's work is cut up, shared by its kernels.
//
// Segments.  Each group's shared prefix is one segment, read with the rows of all its sequences; each
// sequence's own tokens (from its prefix's end to its block's end) are another.  Inside a segment, rows and
// the query heads of one key/value head are packed: packed row m is row m / G, head m % G of the G =
// q_heads / kv_heads that share it, so that keys are read once for all of them.
//
// Units and tiles.  A unit is (segment, key/value head, tile of TM packed rows); it walks its keys in tiles of TK.
// All tiles of all units, in order, are cut into one range of equal cost a block, whatever the lengths are: a block's
// range starts and ends inside units.  Costs are small whole numbers: a tile's (more where a row tile is more than half full
// and the kernel works on its halves in turn) and a unit's own, for setting it up and writing it out.  The part of a
// unit in one block is a piece; it leaves its running
// maximum, sum and weighted values in the workspace, and k_attend_join adds a row's pieces in order.  A unit
// that is one piece and the only one of its rows writes its output itself.
//
// Places are 64 bits wide; a key head's cost within a segment fits 31 (the entry point refuses what could pass that), so that a walk
// divides 32-bit numbers only.
//
// Everything is derived from device arrays inside the call; the host knows bounds only.
#pragma once

#include "sv_code8.cuh"

namespace sv {

constexpr float kLog2e = 1.44269504088896340736f;

// What the cutting has in common with its test on the host.
#define SV_HD __host__ __device__ __forceinline__
// The larger parts of the walk, which a kernel may want out of line (sv_attend_few8.cu): instruction fetches cost it more than calls.
#ifndef SV_WALK_PART
#define SV_WALK_PART SV_HD
#endif

// Row and key tiles of a kernel and what they cost: a key tile, one for more than TM / 2 rows, setting a unit up and writing it out.
struct AttendTiles {
    int TM, TK, tile_cost, tall_cost, unit_cost;
};
constexpr AttendTiles kTilesTall{256, 128, 2, 3, 8};   // of up to 128 rows: the streams take one row tile's key tiles in turn
constexpr AttendTiles kTilesFew{32, 128, 1, 1, 2};        // setting a piece up and writing it out take about two tiles
SV_HD constexpr AttendTiles tiles_few32(int rows) { return {rows, 64, 1, 1, 1}; }
SV_HD constexpr AttendTiles tiles_f32(int rows, int padded_dim) { return {rows, padded_dim == 256 ? 32 : 64, 1, 1, 0}; }

// A unit cut by the ranges of several blocks, left by the block that ends it (only its first piece can): without prefixes
// these are all that has to be joined.  The block that begins it is that of place `at`.
struct AttendTail {
    long long slot;         // of the unit; block c's piece is c * TM further
    long long at, total;    // place of the unit's first tile, cost of the launch
    int cost, tiles;        // of a tile; tiles (0: no such unit)
    int r0, m0, vr, h;
};

// What one launch covers and how it cuts it: segments [s0, s1), row and key tiles, blocks, costs.
struct AttendGeo {
    int s0, s1, TM, TK, blocks;
    int tile_cost, tall_cost, unit_cost;   // of a key tile, of one for more than TM / 2 rows, of a unit
    long long *seg_off;   // [s1 - s0 + 1] place of each segment, in the unit order
    size_t slot0;         // its first workspace slot

    void set(const AttendTiles &t) {
        TM = t.TM;
        TK = t.TK;
        tile_cost = t.tile_cost;
        tall_cost = t.tall_cost;
        unit_cost = t.unit_cost;
    }
};

// Whether a key head's cost fits 31 bits for blocks of up to `rows` packed rows over `slots` tokens.
SV_HD bool tiles_fit(const AttendTiles &t, int64_t rows, int64_t slots) {
    const int64_t units = (rows + t.TM - 1) / t.TM, most = t.unit_cost + (slots + t.TK - 1) / t.TK * t.tall_cost;
    return units * most <= INT32_MAX - 1024;
}

struct AttendArgs {
    KvCache c;
    KvScale sc;                             // of a cache held in 8 bits (no pointers: of the type of q)
    KvBatch bt;
    const char *q;
    char *out;
    int64_t q_row, q_head, o_row, o_head;   // bytes
    int q_heads, G;
    float scale_log2;                       // scale * log2(e)
    const int32_t *group_start, *prefix_len;
    int n_groups;
    float *lse;
    sv_stats *stats;
    long long wait_limit; // cycles after which a wait inside a kernel gives up
    int stuck_stage;      // a ring stage whose copies never count as complete (the self-test of such waits), or -1
    AttendGeo geo;        // of this launch
    // workspace
    struct AttendTail *tails;   // [blocks] the unit that a block ends and an earlier one began
    float *part;          // [slots][head_dim] weighted values of a packed row of a piece
    float2 *part_ml;      // [slots] its maximum (of scale * log2(e) * q.k) and sum
};

// Slots: a piece of unit u in block c starts at unit_slot(u) + c * TM.  Units' slots rise by their rows and
// blocks' by TM, and along the walk either the unit or the block moves on, so pieces never share a slot.
inline size_t attend_slots(int64_t rows, int q_heads, bool prefix, bool own, int TM, int blocks) {
    return (size_t)rows * q_heads * ((prefix ? 1 : 0) + (own ? 1 : 0)) + (size_t)TM * blocks;
}

struct Seg {
    int r0, n;            // its rows
    int table;            // sequence whose page table it reads
    int key0, end;        // its tokens: [key0, end)
    int ctx;              // own segments: cached tokens before the block; prefixes: end
    int packed, tiles_m;  // packed rows; tiles of TM of them
    bool chain;           // row i sees tokens up to ctx + i only
};

// The group of sequence b: the last g with group_start[g] <= b.
SV_HD int group_of(const AttendArgs &a, int b) {
    int lo = 0, hi = a.n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.group_start[mid] <= b) lo = mid;
        else hi = mid;
    }
    return lo;
}

SV_HD int clamp_int(long long x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : (int)x; }

// Segment s, with every device value clamped to what the arrays hold.  `check` reports what had to be.
SV_WALK_PART Seg seg_of(const AttendArgs &a, const AttendGeo &geo, int s, bool check) {
    Seg g;
    const int cap = a.bt.max_pages * a.c.page_size;
    if (s < a.n_groups) {
        const int b0 = clamp_int(a.group_start[s], 0, a.bt.B - 1), b1 = clamp_int(a.group_start[s + 1], b0, a.bt.B);
        const int len = a.prefix_len[s];
        g.r0 = b1 > b0 ? seq_rows(a.bt, b0).r0 : 0;
        int r1 = g.r0;
        if (b1 > b0) {
            const SeqRows last = seq_rows(a.bt, b1 - 1);
            r1 = clamp_int((long long)last.r0 + last.n, g.r0, a.bt.rows);
        }
        g.n = r1 - g.r0;
        g.table = b0;
        g.key0 = 0;
        g.end = clamp_int(len, 0, cap);
        g.ctx = g.end;
        g.chain = false;
#ifdef __CUDA_ARCH__
        if (check && (g.end != len || a.group_start[s] != b0 || a.group_start[s + 1] != b1 || (s == 0 && b0 != 0) ||
                      (s == a.n_groups - 1 && b1 != a.bt.B)))
            report_error(a.stats, SV_ERR_INVALID_ARG, b0);
#endif
    } else {
        const int b = s - a.n_groups;
        const SeqRows sr = seq_rows(a.bt, b);
        const int ctx = a.bt.context_len[b];
        const int start = a.n_groups ? a.prefix_len[group_of(a, b)] : 0;
        g.r0 = sr.r0;
        g.n = sr.n;
        g.table = b;
        g.ctx = clamp_int(ctx, 0, cap);
        g.key0 = clamp_int(start, 0, g.ctx);
        g.end = clamp_int((long long)g.ctx + sr.n, 0, cap);
        g.chain = a.bt.parents == nullptr;
#ifdef __CUDA_ARCH__
        if (check && (!sr.ok || g.ctx != ctx || g.key0 != start || (long long)g.ctx + sr.n > cap))
            report_error(a.stats, SV_ERR_INVALID_ARG, b);
#endif
    }
    g.packed = g.n * a.G;
    g.tiles_m = (g.packed + geo.TM - 1) / geo.TM;
    return g;
}

// One past the last token that row tile t of the segment sees, and its tiles of keys.
SV_HD int seg_end(const AttendArgs &a, const AttendGeo &geo, const Seg &g, int t) {
    if (!g.chain) return g.end;
    const int last = min((t + 1) * geo.TM, g.packed) - 1;
    return min(g.ctx + last / a.G + 1, g.end);
}

SV_HD int seg_tiles(const AttendArgs &a, const AttendGeo &geo, const Seg &g, int t) {
    return (seg_end(a, geo, g, t) - g.key0 + geo.TK - 1) / geo.TK;
}

// Cost of a key tile of row tile t, and of the unit.
SV_HD int tile_cost(const AttendGeo &geo, const Seg &g, int t) {
    return 2 * min(geo.TM, g.packed - t * geo.TM) > geo.TM ? geo.tall_cost : geo.tile_cost;
}
SV_WALK_PART int unit_span(const AttendArgs &a, const AttendGeo &geo, const Seg &g, int t) {
    const int kt = seg_tiles(a, geo, g, t);
    return kt > 0 ? geo.unit_cost + kt * tile_cost(geo, g, t) : 0;
}

// Place of row tile t among a key head's units (t = tiles_m: the cost of all).
SV_WALK_PART int units_before(const AttendArgs &a, const AttendGeo &geo, const Seg &g, int t) {
    if (t <= 0) return 0;
    if (!g.chain) return (t - 1) * unit_span(a, geo, g, 0) + unit_span(a, geo, g, t - 1);   // all but the last are full
    int n = 0;
    for (int u = 0; u < t; ++u) n += unit_span(a, geo, g, u);
    return n;
}

// First workspace slot of unit (h, t) of a segment.
SV_HD size_t unit_slot(const AttendArgs &a, const AttendGeo &geo, const Seg &g, bool prefix, int h, int t) {
    const size_t own = geo.s0 < a.n_groups && !prefix ? (size_t)a.bt.rows * a.q_heads : 0;
    return geo.slot0 + own + (size_t)g.r0 * a.q_heads + (size_t)h * g.packed + (size_t)t * geo.TM;
}

// Ranges of equal cost, the first `more` one longer, of as many blocks as there is a tile's cost for each.
struct Ranges {
    long long each;
    int parts, more;
};

// a / b, both below 2^31 as a rule.  The wide division is kept out of the kernels' code, whose size costs them speed.
__host__ __device__ __noinline__ static long long quotient_wide(long long a, long long b) { return a / b; }
SV_HD long long quotient(long long a, long long b) {
    return ((a | b) >> 31) == 0 ? (long long)((unsigned)a / (unsigned)b) : quotient_wide(a, b);
}

SV_HD Ranges ranges_of(long long total, const AttendGeo &geo) {
    Ranges r{0, 0, 0};
    if (total <= 0) return r;
    r.parts = total >= (long long)geo.blocks * geo.tile_cost ? geo.blocks : max(1, (int)total / geo.tile_cost);
    r.each = quotient(total, r.parts);
    r.more = (int)(total - r.each * r.parts);
    return r;
}

SV_HD long long range_start(const Ranges &r, int c) { return c * r.each + min(c, r.more); }

// The block whose range holds place x.
SV_HD int block_of_place(const Ranges &r, long long x) {
    const long long split = r.more * (r.each + 1);
    return x < split ? (int)quotient(x, r.each + 1) : r.more + (int)quotient(x - split, r.each);
}

// First of a unit's tiles (the first at place `at`, `cost` each) at or after place x.
SV_HD int tile_from(int at, int cost, int tiles, int x) {
    return x <= at ? 0 : min(tiles, (x - at + cost - 1) / cost);
}
// Whether block c holds any.
SV_HD bool block_has(const Ranges &r, int c, long long at, int cost, int tiles) {
    const long long span = (long long)tiles * cost, from = range_start(r, c) - at, to = range_start(r, c + 1) - at;
    return tile_from(0, cost, tiles, (int)(from < 0 ? 0 : from > span ? span : from)) <
           tile_from(0, cost, tiles, (int)(to < 0 ? 0 : to > span ? span : to));
}

// A row's output is complete in its own piece when no prefix adds to it.
SV_HD bool seg_alone(const Seg &g) { return g.key0 == 0; }

struct Piece {
    Seg g;
    int seg, h, t;      // unit
    int vr;             // packed rows of the unit, the first at t * TM
    int k0, k1, kt;     // tiles of keys [k0, k1) of kt
    int at, cost;       // place of the unit's first tile from its key head's, cost of a tile
    int end;            // one past the last token the unit sees
};

// Walks the pieces of one block's range of places, which ends at `stop`.
struct Walk {
    long long head_at, stop, total;   // the key head's place; cost of the launch
    int pos;                          // place from there
    int per_head, h, s;
    Seg g;

    // Takes segment `seg`, whose place is `at`, up at place `first` of it (n its key heads' number).
    SV_HD void begin(const Seg &sg, int seg, int per, long long at, long long first) {
        s = seg;
        g = sg;
        per_head = per;
        h = (int)quotient(first - at, per);
        head_at = at + (long long)h * per;
        pos = (int)(first - head_at);
    }

    SV_HD bool next(const AttendArgs &a, Piece &p) {
        while (head_at + pos < stop) {
            if (pos >= per_head) {   // the next key head, or the next segment's first
                head_at += per_head;
                pos = 0;
                if (per_head == 0 || ++h == a.c.kv_heads) {
                    h = 0;
                    ++s;
                    g = seg_of(a, a.geo, s, false);
                    per_head = units_before(a, a.geo, g, g.tiles_m);
                }
                continue;
            }
            const int lim = stop - head_at < per_head ? (int)(stop - head_at) : per_head;
            p.h = h;
            p.t = 0;
            int unit = 0, span = unit_span(a, a.geo, g, 0);
            if (!g.chain) {
                p.t = min(pos / span, g.tiles_m - 1);
                unit = p.t * span;
                span = unit_span(a, a.geo, g, p.t);
            } else {
                while (pos >= unit + span) {
                    unit += span;
                    span = unit_span(a, a.geo, g, ++p.t);
                }
            }
            p.kt = seg_tiles(a, a.geo, g, p.t);
            p.cost = tile_cost(a.geo, g, p.t);
            p.at = unit + a.geo.unit_cost;
            p.k0 = tile_from(p.at, p.cost, p.kt, pos);
            p.k1 = tile_from(p.at, p.cost, p.kt, lim);
            pos = min(lim, unit + span);
            if (p.k0 >= p.k1) continue;   // the range holds none of the unit's tiles
            p.g = g;
            p.seg = s;
            p.vr = min(a.geo.TM, g.packed - p.t * a.geo.TM);
            p.end = seg_end(a, a.geo, g, p.t);
            return true;
        }
        return false;
    }
};

// A block's tail, from the walk's first piece p (`more` false: it has none).
SV_HD AttendTail tail_of(const AttendArgs &a, const Walk &w, const Piece &p, bool more) {
    AttendTail t{};
    if (more && p.k0 > 0 && p.k1 == p.kt) {
        t.at = w.head_at + p.at;
        t.slot = (long long)unit_slot(a, a.geo, p.g, p.seg < a.n_groups, p.h, p.t);
        t.cost = p.cost;
        t.tiles = p.kt;
        t.total = w.total;
        t.r0 = p.g.r0;
        t.m0 = p.t * a.geo.TM;
        t.vr = p.vr;
        t.h = p.h;
    }
    return t;
}

// The join's view of a segment: its ranges and the key head's place.
struct JoinSeg {
    Seg g;
    Ranges r;
    long long first;
};

SV_HD JoinSeg join_seg(const AttendArgs &a, const AttendGeo &geo, int s, int h) {
    JoinSeg j;
    j.r = ranges_of(geo.seg_off[geo.s1 - geo.s0], geo);
    j.g = seg_of(a, geo, s, false);
    j.first = geo.seg_off[s - geo.s0] + (long long)units_before(a, geo, j.g, j.g.tiles_m) * h;
    return j;
}

// The unit with row tile t: its tiles and the blocks [c0, c1] that may hold pieces of it; c1 < c0: none.
struct JoinUnit {
    long long at;
    int cost, tiles, c0, c1;
};

SV_HD JoinUnit join_unit(const AttendArgs &a, const AttendGeo &geo, const JoinSeg &j, int t) {
    JoinUnit u{0, 1, seg_tiles(a, geo, j.g, t), 0, -1};
    if (u.tiles <= 0 || j.r.parts == 0) return u;
    u.at = j.first + units_before(a, geo, j.g, t) + geo.unit_cost;
    u.cost = tile_cost(geo, j.g, t);
    u.c0 = block_of_place(j.r, u.at);
    u.c1 = block_of_place(j.r, u.at + (long long)(u.tiles - 1) * u.cost);
    return u;
}

// Block-wide: the total cost and, for this block's range, where its walk starts.  Each thread takes a
// run of consecutive segments; warp_sum has THREADS / 32 places.  Block 0 leaves the segments' places for the join and reports bad
// input.
template <int THREADS>
__device__ __forceinline__ void walk_start(const AttendArgs &a, Walk *w, long long *warp_sum) {
    const AttendGeo &geo = a.geo;
    const int NS = geo.s1 - geo.s0;
    const int each = (NS + THREADS - 1) / THREADS;
    const int s0 = min((int)threadIdx.x * each, NS), s1 = min(s0 + each, NS);
    long long mine = 0;
    Seg g{};
    int per = 0;
    for (int s = s0; s < s1; ++s) {
        g = seg_of(a, geo, geo.s0 + s, blockIdx.x == 0);
        per = units_before(a, geo, g, g.tiles_m);
        mine += (long long)per * a.c.kv_heads;
    }
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += v;
    }
    if (lane == 31) warp_sum[wp] = inc;
    __syncthreads();
    long long before = inc - mine, total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < wp) before += warp_sum[i];
        total += warp_sum[i];
    }
    const Ranges r = ranges_of(total, geo);
    const int c = blockIdx.x;
    const long long pos = c < r.parts ? range_start(r, c) : total, stop = c < r.parts ? range_start(r, c + 1) : total;
    if (threadIdx.x == 0) {
        w->total = total;
        w->stop = stop;
        if (pos >= stop) {   // nothing to walk
            w->head_at = stop;
            w->pos = 0;
        }
    }
    if (blockIdx.x == 0 || (pos < stop && pos >= before && pos < before + mine)) {
        long long at = before;
        for (int s = s0; s < s1; ++s) {
            if (each > 1) {   // with one segment a thread, g and per are still those
                g = seg_of(a, geo, geo.s0 + s, false);
                per = units_before(a, geo, g, g.tiles_m);
            }
            const long long n = (long long)per * a.c.kv_heads;
            if (pos < stop && pos >= at && pos < at + n) w->begin(g, geo.s0 + s, per, at, pos);
            if (blockIdx.x == 0) {
                geo.seg_off[s] = at;
                if (s == NS - 1) geo.seg_off[NS] = at + n;
            }
            at += n;
        }
    }
    __syncthreads();
}

// Whether a row sees block token j (both as rows of the block), for a tree: j is the row or an ancestor of it.
// parents[i - 1] < i is checked by the caller that fills the words.
__device__ __forceinline__ void ancestor_words(const int32_t *parents, int i, int n, uint32_t (&w)[(SV_MAX_TREE + 32) / 32],
                                               sv_stats *stats, int b) {
#pragma unroll
    for (int k = 0; k < (SV_MAX_TREE + 32) / 32; ++k) w[k] = 0;
    for (int steps = 0; i >= 0 && steps < n; ++steps) {
#pragma unroll
        for (int k = 0; k < (SV_MAX_TREE + 32) / 32; ++k)
            if ((i >> 5) == k) w[k] |= 1u << (i & 31);
        if (i == 0) break;
        const int p = parents[i - 1];
        if (p < 0 || p >= i) {
            report_error(stats, SV_ERR_INVALID_ARG, b);
            break;
        }
        i = p;
    }
}

// Adds the pieces of the rows that have several.  The launches that made them: of the prefixes' segments (not read without
// groups) and of the own ones; the same where one launch covered both.
cudaError_t launch_attend_join(const AttendArgs &a, const AttendGeo &prefix, const AttendGeo &own, int es, cudaStream_t stream);

// The kernels: float32 arithmetic for any head_dim, in tiles of 64 rows or of kSmallRows, or by warps for up to kFewRows32 packed rows a
// sequence (float32, head_dim <= 128); bf16 with head_dim <= 128 on the tensor cores, a tall form for any number of rows and one for up
// to kFewRows packed rows.  Each fills in a.geo's tiles.
constexpr int kFewRows = 32;
constexpr int kSmallRows = 16;
constexpr int kFewRows32 = 8;
cudaError_t launch_attend_f32(AttendArgs &a, int es, bool small, cudaStream_t stream);
cudaError_t launch_attend_few32(AttendArgs &a, cudaStream_t stream);
cudaError_t launch_attend_tall(AttendArgs &a, cudaStream_t stream);
cudaError_t launch_attend_few(AttendArgs &a, cudaStream_t stream);
cudaError_t launch_attend_few8(AttendArgs &a, cudaStream_t stream);   // launch_attend_few over a cache held in 8 bits

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace sv
