// sv_attend_feed8.cuh — the feed of the tensor-core attention kernels over a cache held in 8 bits: codes come to shared memory as they
// are, and become the bf16 tiles that the products read.
//
// Two warps load, one the keys and one the values: slots of 32 or 64 tokens by TMA boxes (by rows where boxes cannot go) into two rings.
// The four warps that load bf16 caches widen the slots to the products' tiles instead.  There are two kinds of tiles:
//   bf16      a code times its scale, which is a bf16 number: from there on nothing differs, and the result is to the bit that of a
//             bf16 cache of the same values.  A pair of codes takes five instructions (e4m3 to binary16, two of those to float32, a packed
//             product, one to bf16).  For the tall kernel, which the products bound; here.
//   binary16  the code as it is; the scales enter with the scores and the weights.  One instruction a pair.  For few rows, where issue
//             slots and shared memory are near their bounds; sv_attend_few8.cu.
//
// A barrier of a ring is waited for by its phase's parity, so whoever waits for a slot has to wait for each of its fills: with slots that went to
// two warps in turn, one could take the parity of a fill still to come for that of the one before.
#pragma once

#include "sv_attend_feed.cuh"

namespace sv {

constexpr int kRawTokens = 32;    // tokens of a slot of the tall kernel's
constexpr int kMaxSlots8 = 8;

struct Feed8 {
    uint64_t full[2][kMaxSlots8], empty[2][kMaxSlots8];   // of the keys' and the values' slots
    // Scales of the last four tiles (bf16 tiles only).  A loading warp is at most eight slots, two tiles, ahead of the widening ones.
    uint64_t scale_full[2][4];
    uint8_t scale[2][4][kTcKeys];
    uint32_t next[2];                                     // slots a loading warp has begun, left at its end
};

// `readers`: warps that widen a slot.
__device__ __forceinline__ void feed8_init(Feed8 *f8, int slots, int readers) {
    for (int r = 0; r < 2; ++r) {
        for (int i = 0; i < slots; ++i) {
            mbar_init(&f8->full[r][i], 32);
            mbar_init(&f8->empty[r][i], readers);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&f8->scale_full[r][i], 32);
    }
    f8->next[0] = f8->next[1] = 0;
}

// feed_drain's part: boxes on their way to slots.  A loading warp leaves no slot half begun.
template <int SLOTS>
__device__ __noinline__ void feed8_drain(Feed *fd, Feed8 *f8, sv_stats *stats) {
    report_error(stats, SV_ERR_TIMEOUT, -1);
    const long long t0 = clock64();
    for (int r = 0; r < 2; ++r)
        for (uint32_t q = f8->next[r] > SLOTS ? f8->next[r] - SLOTS : 0; q < f8->next[r]; ++q)
            while (!mbar_try_wait_sleep(&f8->full[r][q % SLOTS], (q / SLOTS) & 1, kSuspendHintNs) && clock64() - t0 <= fd->limit) {
            }
}

// Where chunk ch of 16 codes of a slot's token r lies in it: as the TMA swizzle of 128 (64) bytes puts it for tokens of 128 (64) codes, or
// in order.
template <int DP, bool SWIZZLE>
__device__ __forceinline__ int raw_place(int r, int ch) {
    return r * DP + ((!SWIZZLE ? ch : DP == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3)) << 4);
}

// The first token of a lane's box in a tile.  Lanes without a box stay within the tile too: all look pages up tiles ahead, and kMaxSlots leaves room for
// tiles past the last slot, not for 31 boxes of 32 tokens.
SV_HD int box_offset(int lane, int box_rows) { return min(lane * box_rows, kTcKeys - 1); }

// One of the loading warps: kv 0 the keys, 1 the values.  Slots of TOK tokens at raw_base, DP bytes a token.  SCALES: with their scales.  KEYS_SWIZZLED: the
// keys' slots are swizzled.  ALL_BOXES: the last tiles go as boxes too, with what their pages hold past the last token and zeros for pages past it,
// for a softmax that leaves out what a row does not see.
// One warp has to keep up with the others: six cycles an instruction, so a slot's boxes go with as few as can be.  (With the pages of all
// tokens looked up for every tile, as tiles by rows do, it took 4,000 cycles a tile and set the pace.)
template <int DP, int TOK, int SLOTS, bool SCALES, bool KEYS_SWIZZLED, bool ALL_BOXES, bool SPLIT>
__device__ __forceinline__ void feed8_load_as(const AttendArgs &a, const TcArgs &a2, Feed *fd, Feed8 *f8, uint32_t raw_base, int kv, int lane) {
    static_assert(TOK * SLOTS <= 2 * kTcKeys && SLOTS <= kMaxSlots8, "the scales' ring");
    constexpr int SLOT = TOK * DP, NS = kTcKeys / TOK, CH = DP / 16, RPI = 32 / CH;   // slots of a tile; chunks of a token, tokens of a pass by rows
    const int D = a.c.head_dim;
    const CUtensorMap *map = kv ? &a2.v : &a2.k;
    const char *src = kv ? a.c.v : a.c.k;
    const uint8_t *scales = kv ? a.sc.v : a.sc.k;
    uint64_t *const fulls = f8->full[kv], *const empties = f8->empty[kv];
    const int ch = lane % CH, rsub = lane / CH;
    const bool real = ch * 16 < D;   // chunks past the head are zero
    auto raw_at = [&](int r) { return KEYS_SWIZZLED && kv == 0 ? raw_place<DP, true>(r, ch) : raw_place<DP, false>(r, ch); };
    const int psize = a.c.page_size, pshift = a2.page_shift;
    auto page_index = [&](int key) { return pshift >= 0 ? key >> pshift : key / psize; };
    // boxes: a tile's are a lane's each
    const int box_rows = a2.box_rows > 0 ? a2.box_rows : 8, box_token = box_offset(lane, box_rows), my_slot = lane * box_rows / TOK;
    const bool boxes = lane * box_rows < kTcKeys;
    uint32_t slot = 0, parity = 1, begun = 0, tiles = 0;   // the next slot, its empty barrier's parity, slots and tiles begun
    bool on = true;                                        // off once a wait gave up
    auto take = [&]() {   // waits for the next slot
        on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &empties[slot], parity));
        return on;
    };
    auto step = [&]() {
        ++begun;
        if (++slot == SLOTS) {
            slot = 0;
            parity ^= 1;
        }
    };
    for (int it = 0;; ++it) {
        const PieceInfo *pi = &fd->pd[it % kRing];
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1))) break;
        const int k0 = pi->k0, k1 = pi->k1;
        if (k0 >= k1) break;
        const int key0 = pi->key0, end = pi->end, h = pi->h, tab = pi->table;
        const int box_tiles = !ALL_BOXES ? pi->box_tiles : a2.box_rows > 0 && (a2.split || key0 % a2.box_rows == 0) ? INT32_MAX : 0;
        const int32_t *table = a.bt.page_table + tab * a.bt.table_pitch;
        __syncwarp();
        if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
        const uint8_t *my_scales = scales + h * a.sc.head_b;
        // What is loaded ahead is not looked at before it is needed (a warp stops there until it has come), not even to leave it out: past
        // the unit's last token stands that one.
        const int last = end - 1;
        auto box_index = [&](int k) { return page_index(key0 + k * kTcKeys + box_token); };
        auto box_page = [&](int k) { return table[page_index(min(key0 + k * kTcKeys + box_token, last))]; };
        int ahead = box_page(k0);
        // Scales: of the lane's tokens lane, lane + 32, .. of a tile.  Pages are looked up two tiles ahead and scales one.
        int spage[4];
        uint32_t sbyte[4], sgood = 0;   // a bit for each page that is one: the others' scale is 1
        auto ask_pages = [&](int k) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                spage[s] = table[page_index(min(key0 + k * kTcKeys + s * 32 + lane, last))];
            }
        };
        auto ask_scales = [&]() {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const bool good = (unsigned)spage[s] < (unsigned)a.c.n_pages;
                sgood = s == 0 ? good : sgood | (uint32_t)good << s;
                sbyte[s] = my_scales[(good ? spage[s] : 0) * a.sc.page_b];
            }
        };
        if constexpr (SCALES) {
            ask_pages(k0);
            ask_scales();
            ask_pages(k0 + 1);
        }
        for (int k = k0; k < k1 && on; ++k, ++tiles) {
            auto store_scales = [&]() {
                if constexpr (SCALES) {
                    uint8_t *to = f8->scale[kv][tiles & 3] + lane;
#pragma unroll
                    for (int s = 0; s < 4; ++s) to[s * 32] = (sgood >> s) & 1u ? (uint8_t)sbyte[s] : (uint8_t)127;
                    mbar_arrive(&f8->scale_full[kv][tiles & 3]);
                    ask_scales();
                    ask_pages(k + 2);
                }
            };
            if (k < box_tiles) {
                int page = ahead;
                const int place = key0 + k * kTcKeys + box_token - box_index(k) * psize;
                ahead = box_page(k + 1);
                if (ALL_BOXES && key0 + k * kTcKeys + box_token > last) page = a.c.n_pages;   // past the last token: outside the tensor, zeros
                else if (boxes && (unsigned)page >= (unsigned)a.c.n_pages) report_error(a.stats, SV_ERR_INVALID_ARG, tab);
                // split: a box that reaches into the next page goes by rows
                const uint32_t split = SPLIT ? __ballot_sync(0xFFFFFFFFu, boxes && place + 8 > psize) : 0;
#pragma unroll 1
                for (int s = 0; s < NS; ++s) {
                    if (!take()) break;
                    uint64_t *full = &fulls[slot];
                    const uint32_t to = raw_base + slot * SLOT;
                    const uint32_t rows = SPLIT ? (split >> (TOK / 8 * s)) & ((1u << (TOK / 8)) - 1u) : 0;   // boxes of 8 tokens there
                    if (elect_one()) mbar_expect_arrive_n(full, (TOK - 8 * __popc(rows)) * DP, rows ? 0 : 32);
                    __syncwarp();
                    // a bad page id lies outside the tensor and reads zeros
                    if (my_slot == s && !(SPLIT && ((split >> lane) & 1u))) box_load(to + (box_token % TOK) * DP, map, full, 0, h, place, page);
                    __syncwarp();
                    if (SPLIT && rows) {
#pragma unroll 1
                        for (int t0 = 0; t0 < TOK; t0 += 32) {
                            const int key = key0 + k * kTcKeys + s * TOK + t0 + lane, index = page_index(key), id = table[min(index, page_index(last))];
                            const bool good = (unsigned)id < (unsigned)a.c.n_pages && (!ALL_BOXES || key <= last);
                            if (!good && key <= last) report_error(a.stats, SV_ERR_INVALID_ARG, tab);
                            const int64_t off = good ? id * a.c.page_b + (key - index * psize) * a.c.slot_b + h * a.c.head_b : -1;
#pragma unroll 1
                            for (int r0 = 0; r0 < 32; r0 += RPI) {
                                const int r = r0 + rsub;
                                const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
                                const bool ok = o >= 0 && real;
                                if ((rows >> ((t0 + r) >> 3)) & 1u) cp_async16(to + raw_at(t0 + r), src + (ok ? o + ch * 16 : 0), ok);
                            }
                        }
                        cp_async_arrive(full);
                    }
                    step();
                    if (SCALES && s == 0) store_scales();   // after a piece's first boxes
                }
            } else {
                int id[4];   // all pages are asked for before the first is needed
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int key = key0 + k * kTcKeys + s * 32 + lane;
                    id[s] = key < end ? table[page_index(key)] : kNoPage;
                }
#pragma unroll 1
                for (int s = 0; s < NS; ++s) {
                    if (!take()) break;
                    const uint32_t to = raw_base + slot * SLOT;
#pragma unroll 1
                    for (int t0 = 0; t0 < TOK; t0 += 32) {
                        const int key = key0 + k * kTcKeys + s * TOK + t0 + lane, page = id[0];
                        id[0] = id[1];
                        id[1] = id[2];
                        id[2] = id[3];
                        const bool good = (unsigned)page < (unsigned)a.c.n_pages;
                        if (!good && page != kNoPage) report_error(a.stats, SV_ERR_INVALID_ARG, tab);
                        const int64_t off = good ? page * a.c.page_b + (key - page_index(key) * psize) * a.c.slot_b + h * a.c.head_b : -1;
#pragma unroll 2
                        for (int r0 = 0; r0 < 32; r0 += RPI) {
                            const int r = r0 + rsub;
                            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
                            const bool ok = o >= 0 && real;
                            cp_async16(to + raw_at(t0 + r), src + (ok ? o + ch * 16 : 0), ok);
                        }
                    }
                    cp_async_arrive(&fulls[slot]);
                    step();
                    if (SCALES && s == 0) store_scales();
                }
            }
        }
    }
    cp_async_commit();
    cp_async_wait<0>();   // no row is in flight when the block ends; boxes are when a wait gave up
    if (lane == 0) f8->next[kv] = begun;
}

template <int DP, int TOK, int SLOTS, bool SCALES, bool KEYS_SWIZZLED, bool ALL_BOXES>
__device__ __forceinline__ void feed8_load(const AttendArgs &a, const TcArgs &a2, Feed *fd, Feed8 *f8, uint32_t raw_base, int kv, int lane) {
    if (a2.split) feed8_load_as<DP, TOK, SLOTS, SCALES, KEYS_SWIZZLED, ALL_BOXES, true>(a, a2, fd, f8, raw_base, kv, lane);
    else feed8_load_as<DP, TOK, SLOTS, SCALES, KEYS_SWIZZLED, ALL_BOXES, false>(a, a2, fd, f8, raw_base, kv, lane);
}

// 16 codes times their scale as 16 bf16 numbers, two chunks of 16 bytes.
__device__ __forceinline__ void widen16(uint4 w, f32x2 scale, uint32_t (&lo)[4], uint32_t (&hi)[4]) {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = codes4(in[i]);
        float x, y, z, t;
        f2_unpack(f2_mul(f2_pack(f.x, f.y), scale), x, y);
        f2_unpack(f2_mul(f2_pack(f.z, f.w), scale), z, t);
        uint32_t *to = i < 2 ? lo : hi;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(to[(i & 1) * 2]) : "f"(y), "f"(x));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(to[(i & 1) * 2 + 1]) : "f"(t), "f"(z));
    }
}

// Which 16 codes a lane of a widening warp takes in a pass.  Eight lanes take two neighbouring tokens, four chunks each, of a token of 128
// different halves: neither the loads nor the stores to the swizzled tile then meet in a bank.
template <int DP>
struct WidenLane {
    static constexpr int PASS = DP == 128 ? 4 : 8;   // tokens of a pass
    int row0, ch;                                    // its token of the first pass, its chunk
    __device__ __forceinline__ explicit WidenLane(int lane) {
        const int j = lane & 7, p = lane >> 3;
        row0 = DP == 128 ? (p >> 1) * 2 + (j >> 2) : p * 2 + (j >> 2);
        ch = DP == 128 ? (j & 3) + 4 * ((j >> 2) ^ (p & 1)) : j & 3;
    }
};

// One of the four widening warps, bf16 tiles: it also copies its quarter of the query tiles.  Stages at kv_base as feed_produce fills them; a
// stage is full when its two warps have arrived.
template <int DP, int STAGES, int QROWS, int SLOTS>
__device__ __forceinline__ void feed8_widen(const AttendArgs &a, Feed *fd, Feed8 *f8, uint32_t q_base, uint32_t kv_base, uint32_t raw_base, int wl,
                                            int lane) {
    constexpr int TILE = 128 * DP * 2, HALF = 128 * 128, SLOT = kRawTokens * DP;
    const int D = a.c.head_dim, kv = wl >> 1, sub = wl & 1;
    raw_base += kv * SLOTS * SLOT;
    const WidenLane<DP> me(lane);
    const int row0 = me.row0, ch = me.ch;
    constexpr int PASS = WidenLane<DP>::PASS;
    const uint32_t from = row0 * DP + ch * 16, to_half = (ch >> 2) * HALF;
    uint32_t seq = kv, q_phases = 0, slots = 0, tiles = 0;   // slots: the next of its ring
    int qnext = 0;
    bool on = true;
    for (int it = 0;; ++it) {
        const PieceInfo *pi = &fd->pd[it % kRing];
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1))) break;
        const int k0 = pi->k0, k1 = pi->k1;
        if (k0 >= k1) break;
        const int vr = pi->vr, h = pi->h, m0 = pi->m0, r0 = pi->r0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
        const bool two = vr > QROWS;   // two row tiles share the keys
        for (int t = 0; t < (two ? 2 : 1) && on; ++t) {   // queries, a quarter of the tile a warp
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
            const int qch = lane & 7, rsub = lane >> 3;
#pragma unroll 2
            for (int pass = 0; pass < QROWS / 16; ++pass) {
                const int r = pass * 4 + rsub;
                const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
#pragma unroll
                for (int half = 0; half < DP / 64; ++half) {
                    const bool ok = o >= 0 && half * 64 + qch * 8 < D;
                    cp_async16(qtile + half * (QROWS * 128) + (wl * (QROWS / 4) + r) * 128 + ((qch ^ (r & 7)) << 4),
                               a.q + (ok ? o + (half * 64 + qch * 8) * 2 : 0), ok);
                }
            }
            cp_async_arrive(&fd->q_full[qs]);
        }
        if (!two) qnext ^= 1;
        for (int k = k0; k < k1 && on; ++k, ++tiles) {
            const uint32_t stage = seq % STAGES;
            on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &fd->kv_empty[stage], ((seq / STAGES) & 1) ^ 1) &&
                                             wait_phase(fd, &f8->scale_full[kv][tiles & 3], (tiles >> 2) & 1));
            if (!on) break;
            seq += 2;
            const volatile uint8_t *bytes = f8->scale[kv][tiles & 3];
#pragma unroll 1
            for (int s = 0; s < 4 && on; ++s, ++slots) {   // each warp half of a slot
                const uint32_t slot = slots % SLOTS;
                on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &f8->full[kv][slot], (slots / SLOTS) & 1));
                if (!on) break;
                const uint32_t raw = raw_base + slot * SLOT + from;
                const uint32_t tile = kv_base + stage * TILE + s * (kRawTokens * 128) + to_half;
#pragma unroll
                for (int v = 0; v < kRawTokens / PASS / 2; ++v) {
                    const int u = sub * (kRawTokens / PASS / 2) + v, row = u * PASS + row0;
                    uint4 w;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                 : "r"(raw + u * (PASS * DP)));
                    const float f = scale_of(bytes[s * kRawTokens + row]);
                    uint32_t lo[4], hi[4];
                    widen16(w, f2_pack(f, f), lo, hi);
                    const int c = 2 * (ch & 3);
                    sts128(tile + row * 128 + ((c ^ (row & 7)) << 4), lo);
                    sts128(tile + row * 128 + (((c + 1) ^ (row & 7)) << 4), hi);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&f8->empty[kv][slot]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&fd->kv_full[stage]);
        }
    }
    cp_async_commit();
    cp_async_wait<0>();
}

// Element d of head h's value at byte offset `off` (head 0) of page `page`, as the tile holds it.
template <bool C8>
__device__ __forceinline__ float cached_value(const AttendArgs &a, int64_t off, const int32_t *table, int key, int h, int d) {
    const char *v = a.c.v + off + h * a.c.head_b;
    if constexpr (C8) {
        const float f = scale_of(a.sc.v[table[key / a.c.page_size] * a.sc.page_b + h * a.sc.head_b]);
        float x = codes2(reinterpret_cast<const uint8_t *>(v)[d]).x * f;
        uint16_t b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(x));
        return __uint_as_float((uint32_t)b << 16);
    } else {
        return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(v)[d] << 16);
    }
}

inline bool cache_map8(CUtensorMap *map, char *base, const KvCache &c, int width, int box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.kv_heads, (cuuint64_t)c.page_size, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.head_b, (cuuint64_t)c.slot_b, (cuuint64_t)c.page_b};
    const cuuint32_t box[4] = {(cuuint32_t)width, 1, (cuuint32_t)box_rows, 1}, one[4] = {1, 1, 1, 1};
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// tc_args for codes: boxes of up to a slot's 32 tokens by whole heads.
inline TcArgs tc_args8(const KvCache &c, int width, bool keys_swizzled, uint32_t shape_s) {
    TcArgs t{};
    t.shape_s = shape_s;
    const int ps = c.page_size;
    t.page_shift = (ps & (ps - 1)) == 0 ? __builtin_ctz(ps) : -1;
    const int rows = ps % 32 == 0 ? 32 : ps % 16 == 0 ? 16 : ps >= 8 ? 8 : 0;
    t.split = rows == 8 && ps % 8 != 0;
    if (rows > 0) {
        t.box_rows = rows;
        const CUtensorMapSwizzle none = CU_TENSOR_MAP_SWIZZLE_NONE, own = width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
        if (encode_tiled() == nullptr || !cache_map8(&t.k, c.k, c, width, rows, keys_swizzled ? own : none) || !cache_map8(&t.v, c.v, c, width, rows, none))
            t.box_rows = 0;
    }
    return t;
}

}  // namespace sv
