// sv_attend_feed.cuh — what the tensor-core kernels of sv_kv_attend share: the walk that describes a block's pieces, the
// producer warps that gather keys, values and queries from their pages into swizzled shared memory, bounded waits.
//
// Ring.  Stages of 128 tokens (keys, then values of a tile, in turn) are filled by two producer warps each and freed by the commit of
// the product that read them.
#pragma once

#include "sv_attend.cuh"
#include "sv_tc.cuh"

namespace sv {

constexpr int kTcThreads = 512;       // four warpgroups: two of softmax, producers, products and the walk
constexpr int kTcKeys = 128;          // tokens of a tile
constexpr int kRing = 3;              // piece descriptions in flight
constexpr int kNoPage = INT32_MIN;    // a token past the unit's last
// Registers: 256 softmax threads take 176, the other 256 give down to 80; 512 x 128 at launch.
constexpr int kRegsSoftmax = 176, kRegsOther = 80;

struct PieceInfo {
    long long slot;                   // first workspace slot
    int r0, m0, vr, h;                // segment's first row, first packed row, rows, key head
    int table, key0, ctx, end;        // page table's sequence, tokens
    int k0, k1;                       // key tiles; k0 == k1: no more pieces
    uint32_t seq;                     // ring number of the first tile's keys
    int box_tiles;                    // tiles before this one load as boxes, the others by rows
    bool own, tree, whole;            // own segment, tree mask, output complete here
    uint8_t par[SV_MAX_TREE];         // a tree's parents (255: invalid)
};

struct Feed {
    uint64_t kv_full[8], kv_empty[8], q_full[2], q_empty[2], pd_full[kRing], pd_empty[kRing];
    PieceInfo pd[kRing];
    uint32_t vflag[8][4];             // per stage: tokens whose values are not finite (tiles with hidden tokens only)
    uint32_t tmem;
    int dead;                         // a wait gave up: nobody waits for data any more
    long long limit;                  // cycles after which one does
    uint32_t next[4];                 // a producer warp's next ring number, left at its end
};

// Waits for a phase; false when it gave up, which one wait does after the limit and from then on every one whose phase has not
// completed.  The block runs to its end with meaningless results: the producers stop, the products and the softmax go on over the
// same pieces (its warps meet at barriers, which all have to reach), and feed_drain waits for the copies in flight.  Only
// descriptions of pieces are still waited for (`patient`): they come from the walk, which waits for nothing but their readers, so
// that all warps see the same pieces to the last.  A tile then takes microseconds, and that wait's own limit of many seconds is
// never met.
template <bool patient = false>
__device__ __forceinline__ bool wait_phase(Feed *fd, uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long until = clock64() + (patient ? 8 * kWaitLimitCycles : fd->limit);
    do {
        if (!patient && *reinterpret_cast<volatile int *>(&fd->dead)) return false;
        if (clock64() > until) {
            *reinterpret_cast<volatile int *>(&fd->dead) = 1;   // reported at the block's end: less code at every wait
            return false;
        }
    } while (!mbar_try_wait_sleep(bar, parity, kSuspendHintNs));
    return true;
}

// `readers`: warps that read a piece description.
__device__ __forceinline__ void feed_init(Feed *fd, const AttendArgs &a, int readers) {
    for (int i = 0; i < 8; ++i) {
        mbar_init(&fd->kv_full[i], i == a.stuck_stage ? 65 : 64);
        mbar_init(&fd->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(&fd->q_full[i], 128);
        mbar_init(&fd->q_empty[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
        mbar_init(&fd->pd_full[i], 1);
        mbar_init(&fd->pd_empty[i], readers);
    }
    fd->dead = 0;
    fd->limit = a.wait_limit;
    for (int i = 0; i < 4; ++i) fd->next[i] = i >> 1;
}

// After a wait gave up, by one thread when every warp is done: reports it and waits for the boxes that are still on their way to
// shared memory, which the next block will use.  Ring number q is filled by two warps; one that had stopped is stood in for.  A
// stage is filled again only after its last fill was complete, so only the last one counts.
template <int STAGES>
__device__ __noinline__ void feed_drain(Feed *fd, sv_stats *stats) {
    report_error(stats, SV_ERR_TIMEOUT, -1);
    const long long t0 = clock64();
    const int end = (int)max(max(fd->next[0], fd->next[1]), max(fd->next[2], fd->next[3]));   // ring numbers begun are below
    for (int last = end - 1; last >= 0 && last >= end - STAGES; --last) {
        for (int q = last; q >= 0; q -= STAGES) {
            const int pair = (q & 1) * 2;
            const bool first = q < (int)fd->next[pair], second = q < (int)fd->next[pair + 1];
            if (!first && !second) continue;
            uint64_t *bar = &fd->kv_full[q % STAGES];
            if (first != second) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 32;" ::"r"(smem_addr(bar)) : "memory");
            while (!mbar_try_wait_sleep(bar, (q / STAGES) & 1, kSuspendHintNs) && clock64() - t0 <= fd->limit) {
            }
            break;
        }
    }
}

__device__ __forceinline__ bool not_finite16(uint4 w) {
    auto bad = [](uint32_t x) { return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u; };
    return bad(w.x) || bad(w.y) || bad(w.z) || bad(w.w);
}

// The barrier gets this thread's arrival once its copies so far have landed.  The copies are ordinary writes to shared memory: who
// waits for the barrier fences them (fence_async_smem) before the tensor cores read them.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// `bytes` more to come, and n arrivals.
__device__ __forceinline__ void mbar_expect_arrive_n(uint64_t *bar, uint32_t bytes, uint32_t n) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
    if (n) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t at, const uint32_t (&x)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
}

__device__ __forceinline__ f32x2 f2_mul(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two weights as bf16 pairs: the upper parts are cut off, the lower ones are the rounded rest, 16 bits in all (within 2^-16).
// Both parts of a weight above 0 are above 0 (to 2^-102; the rest is taken from hi (1 - 2^-24), one instruction as it is from
// hi): an infinite value times the two then adds up to that infinity.  With a rounded upper part the lower one is 0 or negative for
// half of the weights, and the sum was NaN.
__device__ __forceinline__ void weight_parts(f32x2 e, uint32_t &hi, uint32_t &lo) {
    float a, b;
    f2_unpack(e, a, b);
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    f2_unpack(f2_fma(f2_from_bf16x2(hi), f2_pack(-0x1.fffffep-1f, -0x1.fffffep-1f), e), a, b);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(b), "f"(a));
}

// Values of a tile with hidden tokens, by 128 threads: thread t looks at token t.  A token whose values are not all finite becomes
// zeros, so that 0 * inf of a row that does not see it cannot reach the output, and its bit is set in flags[t / 32].
template <int DP>
__device__ __forceinline__ void scan_values(uint32_t tile, int t, uint32_t *flags) {
    uint4 w[DP / 8];
    bool bad = false;
#pragma unroll
    for (int ch = 0; ch < DP / 8; ++ch) {
        const uint32_t at = tile + (ch >> 3) * (128 * 128) + t * 128 + (((ch & 7) ^ (t & 7)) << 4);
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[ch].x), "=r"(w[ch].y), "=r"(w[ch].z), "=r"(w[ch].w) : "r"(at));
    }
#pragma unroll
    for (int ch = 0; ch < DP / 8; ++ch) bad |= not_finite16(w[ch]);
    if (bad) {
        const uint32_t zero[4] = {0, 0, 0, 0};
        for (int ch = 0; ch < DP / 8; ++ch) sts128(tile + (ch >> 3) * (128 * 128) + t * 128 + (((ch & 7) ^ (t & 7)) << 4), zero);
    }
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, bad);
    if ((t & 31) == 0) flags[t >> 5] = all;
    fence_async_smem();
}

// Keys and values as 4-D tensors (element, head, slot, page) with boxes of 64 elements by box_rows slots, loaded with the
// 128-byte swizzle.  Where the page size is no multiple of 8 (split), boxes of 8 whose slots lie in two pages are copied by rows;
// box_rows is 0, and everything goes by rows, where a page has fewer than 8 slots.
struct TcArgs {
    CUtensorMap k, v;
    int box_rows, split;
    int page_shift;       // log2(page_size), or -1
    uint32_t shape_s;     // of the score product
};

// The producers' part, a warp of four.  QROWS rows a query tile; query tiles at q_base, stages at kv_base.  Two warps load the keys and
// two the values; of a pair, each takes 64 elements of all 128 tokens (heads of 128), or 64 tokens.  A warp so waits for one
// stage a tile and issues its boxes in one go: with the four sharing every stage, 32 tokens each, the producers set the pace.
template <int DP, int STAGES, int QROWS, bool SPLIT>
__device__ __forceinline__ void feed_produce_as(const AttendArgs &a, const TcArgs &a2, Feed *fd, uint32_t q_base, uint32_t kv_base, int wl,
                                                int lane) {
    constexpr int TILE = 128 * DP * 2, HALF = 128 * 128;
    constexpr int ROWS = DP == 128 ? 128 : 64;   // tokens of a warp
    const int D = a.c.head_dim, kv = wl >> 1, sub = wl & 1;
    const int row0 = DP == 128 ? 0 : sub * 64, col0 = DP == 128 ? sub * 64 : 0;   // its tokens and elements of a tile
    const uint32_t part = DP == 128 ? sub * HALF : sub * 64 * 128;               // where they are
    const CUtensorMap *map = kv ? &a2.v : &a2.k;
    const char *src = kv ? a.c.v : a.c.k;
    const int ch = lane & 7, rsub = lane >> 3;   // rows go four at a time, 8 chunks of 16 bytes each
    const bool real = col0 + ch * 8 < D;         // chunks past the head are zero
    const int psize = a.c.page_size, pshift = a2.page_shift;
    auto page_index = [&](int key) { return pshift >= 0 ? key >> pshift : key / psize; };
    uint32_t seq = kv, q_phases = 0;   // q_phases: a bit a query tile
    int qnext = 0;
    bool on = true;                    // off once a wait gave up
    for (int it = 0;; ++it) {
        const PieceInfo *pi = &fd->pd[it % kRing];
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1))) break;
        const int k0 = pi->k0, k1 = pi->k1;
        if (k0 >= k1) break;
        const int vr = pi->vr, key0 = pi->key0, end = pi->end, h = pi->h, m0 = pi->m0, r0 = pi->r0, tab = pi->table;
        const int box_tiles = pi->box_tiles, boxes = box_tiles > 0 ? ROWS / a2.box_rows : 0;
        const int32_t *table = a.bt.page_table + tab * a.bt.table_pitch;
        __syncwarp();
        if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
        const bool two = vr > QROWS;   // two row tiles share the keys
        auto by_box = [&](int k) { return k < box_tiles; };
        // this lane's box of a tile, as (page, slot); fetched a tile ahead
        auto box_key = [&](int k) { return key0 + k * kTcKeys + row0 + lane * a2.box_rows; };
        auto box_page = [&](int k) { return k < k1 && by_box(k) && lane < boxes ? table[page_index(box_key(k))] : kNoPage; };
        int page = box_page(k0);
        for (int k = k0; k < k1 && on; ++k) {
            const int pg = page;
            page = box_page(k + 1);
            const uint32_t stage = seq % STAGES;
            const uint32_t tile = kv_base + stage * TILE + part;
            // Products that gave a wait up free stages that are still being filled: nothing is copied any more from then on.
            on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &fd->kv_empty[stage], ((seq / STAGES) & 1) ^ 1) &&
                                             !*reinterpret_cast<volatile int *>(&fd->dead));
            if (!on) break;
            seq += 2;
            if (by_box(k)) {
                const int key = box_key(k), slot = key - page_index(key) * psize;
                if ((unsigned)pg >= (unsigned)a.c.n_pages && pg != kNoPage) report_error(a.stats, SV_ERR_INVALID_ARG, tab);
                // split: a box that reaches into the next page goes by rows
                const uint32_t split = SPLIT ? __ballot_sync(0xFFFFFFFFu, lane < boxes && slot + 8 > psize) : 0;
                if (elect_one()) mbar_expect_arrive_n(&fd->kv_full[stage], (ROWS - 8 * __popc(split)) * 128, split ? 0 : 32);
                __syncwarp();
                // a bad page id lies outside the tensor and reads zeros
                if (lane < boxes && !((split >> lane) & 1u)) box_load(tile + lane * a2.box_rows * 128, map, &fd->kv_full[stage], col0, h, slot, pg);
                __syncwarp();
                if (split) {
                    int pg2 = 0;
                    if ((split >> lane) & 1u) {
                        pg2 = table[page_index(key) + 1];
                        if ((unsigned)pg2 >= (unsigned)a.c.n_pages) report_error(a.stats, SV_ERR_INVALID_ARG, tab);
                    }
#pragma unroll 1
                    for (uint32_t left = split; left; left &= left - 1) {
                        const int b = __ffs(left) - 1, s0 = __shfl_sync(0xFFFFFFFFu, slot, b);
                        const int p0 = __shfl_sync(0xFFFFFFFFu, pg, b), p1 = __shfl_sync(0xFFFFFFFFu, pg2, b);
#pragma unroll 1
                        for (int r = rsub; r < 8; r += 4) {
                            const bool over = s0 + r >= psize;
                            const int id = over ? p1 : p0, sl = over ? s0 + r - psize : s0 + r;
                            const bool ok = (unsigned)id < (unsigned)a.c.n_pages && real;
                            const int64_t o = id * a.c.page_b + sl * a.c.slot_b + h * a.c.head_b + (col0 + ch * 8) * 2;
                            cp_async16(tile + (b * 8 + r) * 128 + ((ch ^ r) << 4), src + (ok ? o : 0), ok);
                        }
                    }
                    cp_async_arrive(&fd->kv_full[stage]);
                }
            } else {
                // Not unrolled: the block's five kinds of warps share the instruction cache, and these loops laid out in full
                // cost the whole kernel a seventh of its speed.
                int id[ROWS / 32];   // all pages are asked for before the first is needed
#pragma unroll
                for (int i = 0; i < ROWS / 32; ++i) {
                    const int key = key0 + k * kTcKeys + row0 + i * 32 + lane;
                    id[i] = key < end ? table[page_index(key)] : kNoPage;
                }
#pragma unroll 1
                for (int i = 0; i < ROWS / 32; ++i) {
                    const int key = key0 + k * kTcKeys + row0 + i * 32 + lane;
                    int64_t off = -1;
                    if ((unsigned)id[0] < (unsigned)a.c.n_pages)
                        off = id[0] * a.c.page_b + (key - page_index(key) * psize) * a.c.slot_b + h * a.c.head_b;
                    else if (id[0] != kNoPage)
                        report_error(a.stats, SV_ERR_INVALID_ARG, tab);
#pragma unroll
                    for (int j = 0; j + 1 < ROWS / 32; ++j) id[j] = id[j + 1];
#pragma unroll 2
                    for (int p = 0; p < 8; ++p) {
                        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, p * 4 + rsub);
                        const bool ok = o >= 0 && real;
                        const int r = row0 + i * 32 + p * 4 + rsub;   // r & 7 is the swizzle
                        cp_async16(tile + (i * 32 + p * 4 + rsub) * 128 + ((ch ^ (r & 7)) << 4), src + (ok ? o + (col0 + ch * 8) * 2 : 0), ok);
                    }
                }
                cp_async_arrive(&fd->kv_full[stage]);
            }
            if (k == k0) {   // queries, a quarter of the tile a warp; after the first keys, which memory has to bring
                for (int t = 0; t < (two ? 2 : 1); ++t) {
                    const int qs = two ? t : qnext;
                    on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &fd->q_empty[qs], ((q_phases >> qs) & 1) ^ 1));
                    if (!on) break;
                    q_phases ^= 1u << qs;
                    const int m = t * QROWS + wl * (QROWS / 4) + lane;
                    int64_t off = -1;
                    if (lane < QROWS / 4 && m < vr) {
                        const int r = (m0 + m) / a.G;
                        off = (int64_t)(r0 + r) * a.q_row + (int64_t)(h * a.G + (m0 + m - r * a.G)) * a.q_head;
                    }
                    const uint32_t qtile = q_base + qs * (QROWS * DP * 2);
#pragma unroll 2
                    for (int p = 0; p < QROWS / 16; ++p) {
                        const int r = p * 4 + rsub;
                        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
#pragma unroll
                        for (int half = 0; half < DP / 64; ++half) {
                            const bool ok = o >= 0 && half * 64 + ch * 8 < D;
                            cp_async16(qtile + half * (QROWS * 128) + (wl * (QROWS / 4) + r) * 128 + ((ch ^ (r & 7)) << 4),
                                       a.q + (ok ? o + (half * 64 + ch * 8) * 2 : 0), ok);
                        }
                    }
                    cp_async_arrive(&fd->q_full[qs]);
                }
                if (!two) qnext ^= 1;
            }
        }
    }
    cp_async_commit();
    cp_async_wait<0>();   // no row is in flight when the block ends; boxes are when a wait gave up
    if (lane == 0) fd->next[wl] = seq;
}

// Two copies of the loop: with the code for split boxes in it, pages without them took 595 us instead of 545 (512 x 6 rows over 1-2k
// tokens; the instruction cache again).
template <int DP, int STAGES, int QROWS>
__device__ __forceinline__ void feed_produce(const AttendArgs &a, const TcArgs &a2, Feed *fd, uint32_t q_base, uint32_t kv_base, int wl,
                                             int lane) {
    if (a2.split) feed_produce_as<DP, STAGES, QROWS, true>(a, a2, fd, q_base, kv_base, wl, lane);
    else feed_produce_as<DP, STAGES, QROWS, false>(a, a2, fd, q_base, kv_base, wl, lane);
}

// The walk's part, one warp: describes the pieces, then that there are no more.
__device__ __forceinline__ void feed_walk(const AttendArgs &a, const TcArgs &a2, Feed *fd, Walk w, int lane) {
    uint32_t seq = 0;
    for (int it = 0;; ++it) {
        Piece p;
        const bool more = w.next(a, p);
        if (it == 0 && lane == 0) a.tails[blockIdx.x] = tail_of(a, w, p, more);
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(fd, &fd->pd_empty[it % kRing], ((it / kRing) & 1) ^ 1))) break;
        PieceInfo *pi = &fd->pd[it % kRing];
        const bool own = more && p.seg >= a.n_groups, tree = own && a.bt.parents != nullptr;
        if (more && tree) {
            const int32_t *par = a.bt.parents + (int64_t)p.g.table * (a.bt.n - 1);
            for (int j = lane; j < a.bt.n - 1; j += 32) {
                const int v = par[j];
                const bool ok = v >= 0 && v <= j;
                if (!ok) report_error(a.stats, SV_ERR_INVALID_ARG, p.g.table);
                pi->par[j] = ok ? (uint8_t)v : (uint8_t)255;
            }
        }
        if (lane == 0) {
            if (more) {
                pi->slot = (long long)(unit_slot(a, a.geo, p.g, !own, p.h, p.t) + (size_t)blockIdx.x * a.geo.TM);
                pi->r0 = p.g.r0;
                pi->m0 = p.t * a.geo.TM;
                pi->vr = p.vr;
                pi->h = p.h;
                pi->table = p.g.table;
                pi->key0 = p.g.key0;
                pi->ctx = p.g.ctx;
                pi->end = p.end;
                // a tile that every row sees whole goes as boxes where no box would cross a page
                pi->box_tiles = a2.box_rows > 0 && (a2.split || p.g.key0 % a2.box_rows == 0) ? ((own ? p.g.ctx : p.end) - p.g.key0) / kTcKeys : 0;
                pi->k0 = p.k0;
                pi->k1 = p.k1;
                pi->seq = seq;
                pi->own = own;
                pi->tree = tree;
                pi->whole = p.k0 == 0 && p.k1 == p.kt && own && seg_alone(p.g);
            } else {
                pi->k0 = pi->k1 = 0;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&fd->pd_full[it % kRing]);
        if (more) seq += 2 * (p.k1 - p.k0);
        else break;
    }
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &res) != cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

inline bool cache_map(CUtensorMap *map, char *base, const KvCache &c, int box_rows) {
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.kv_heads, (cuuint64_t)c.page_size, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.head_b, (cuuint64_t)c.slot_b, (cuuint64_t)c.page_b};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1}, one[4] = {1, 1, 1, 1};
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tensors of a call.  Boxes of up to 64 slots, whole swizzle groups of 8 rows, that never cross a page.  512 x 6 rows over 1-2k
// tokens: in pages of 8 to 64 slots 541-552 us, of 24 561, of 100 609; copied by rows 816, as pages of fewer than 8 slots are.
inline TcArgs tc_args(const KvCache &c, uint32_t shape_s) {
    TcArgs t{};
    t.shape_s = shape_s;
    const int ps = c.page_size;
    t.page_shift = (ps & (ps - 1)) == 0 ? __builtin_ctz(ps) : -1;
    const int rows = ps % 64 == 0 ? 64 : ps % 32 == 0 ? 32 : ps % 16 == 0 ? 16 : ps >= 8 ? 8 : 0;
    t.split = rows == 8 && ps % 8 != 0;
    if (rows > 0) {
        t.box_rows = rows;
        if (encode_tiled() == nullptr || !cache_map(&t.k, c.k, c, t.box_rows) || !cache_map(&t.v, c.v, c, t.box_rows)) t.box_rows = 0;
    }
    return t;
}

}  // namespace sv
