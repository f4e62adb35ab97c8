// sv_attend_feed8.cuh — the feed of the tensor-core attention kernels over a cache held in 8 bits: codes come to shared memory as they
// are, and become the bf16 tiles that the products read.
//
// Two warps load, one the keys and one the values: slots of 32 tokens by TMA boxes (by rows where boxes cannot go), with
// the tokens' scales, into two rings.  The four warps that load bf16 caches turn the slots into tiles instead, two for the keys and
// two for the values, every other slot each: a code times its scale is a bf16 number, so from there on nothing differs, and the result
// is to the bit that of a bf16 cache of the same values.
//
// A pair of codes takes five instructions (e4m3 to binary16, two of those to float32, a packed product, one to bf16), 640 a
// lane and pair of tiles of 128 x 128: as much as the softmax, and both fit under the 1,450 cycles that a pair takes at an SM's
// share of the measured copy bandwidth.
#pragma once

#include "sv_attend_feed.cuh"

namespace sv {

constexpr int kRawTokens = 32;    // tokens of a slot
constexpr int kMaxSlots8 = 12;

struct Feed8 {
    uint64_t full[2][kMaxSlots8], empty[2][kMaxSlots8];   // of the keys' and the values' slots
    float scale[2][kMaxSlots8][kRawTokens];
    uint32_t next[2];                                     // slots a loading warp has begun, left at its end
};

__device__ __forceinline__ void feed8_init(Feed8 *f8, int slots) {
    for (int r = 0; r < 2; ++r)
        for (int i = 0; i < slots; ++i) {
            mbar_init(&f8->full[r][i], 2 * 32);   // each lane once for its copies and once for its token's scale
            mbar_init(&f8->empty[r][i], 1);
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

// One of the loading warps: kv 0 the keys, 1 the values.  Slots at raw_base, DP bytes a token.
template <int DP, int SLOTS, bool SPLIT>
__device__ __forceinline__ void feed8_load_as(const AttendArgs &a, const TcArgs &a2, Feed *fd, Feed8 *f8, uint32_t raw_base, int kv, int lane) {
    constexpr int SLOT = kRawTokens * DP, CH = DP / 16, RPI = 32 / CH;   // chunks of a token, tokens of a pass by rows
    const int D = a.c.head_dim;
    const CUtensorMap *map = kv ? &a2.v : &a2.k;
    const char *src = kv ? a.c.v : a.c.k;
    const uint8_t *scales = kv ? a.sc.v : a.sc.k;
    const int ch = lane % CH, rsub = lane / CH;
    const bool real = ch * 16 < D;   // chunks past the head are zero
    const int psize = a.c.page_size, pshift = a2.page_shift;
    auto page_index = [&](int key) { return pshift >= 0 ? key >> pshift : key / psize; };
    uint32_t q = 0;                  // slots begun
    bool on = true;                  // off once a wait gave up
    // A slot's scales are asked for with its tokens and stored when the next slot is begun, or before a wait.
    uint32_t held = 0, held_slot = 0;
    bool holds = false;
    auto store_scale = [&]() {
        if (holds) {
            f8->scale[kv][held_slot][lane] = scale_of(held);
            mbar_arrive(&f8->full[kv][held_slot]);
            holds = false;
        }
    };
    for (int it = 0;; ++it) {
        const PieceInfo *pi = &fd->pd[it % kRing];
        if (!mbar_test_wait(&fd->pd_full[it % kRing], (it / kRing) & 1)) store_scale();
        __syncwarp();
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1))) break;
        const int k0 = pi->k0, k1 = pi->k1;
        if (k0 >= k1) break;
        const int key0 = pi->key0, end = pi->end, h = pi->h, tab = pi->table, box_tiles = pi->box_tiles;
        const int boxes = box_tiles > 0 ? kRawTokens / a2.box_rows : 0;
        const int32_t *table = a.bt.page_table + tab * a.bt.table_pitch;
        __syncwarp();
        if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
        const uint8_t *my_scales = scales + h * a.sc.head_b;
        // the pages of this lane's tokens of a tile, asked for a tile ahead
        int ahead[4];
        auto ask = [&](int k) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int key = key0 + k * kTcKeys + s * kRawTokens + lane;
                ahead[s] = k < k1 && key < end ? table[page_index(key)] : kNoPage;
            }
        };
        ask(k0);
        store_scale();   // of the last piece's last slot, while the pages come
        for (int k = k0; k < k1 && on; ++k) {
            int id[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) id[s] = ahead[s];
            ask(k + 1);
#pragma unroll 1
            for (int s = 0; s < 4; ++s) {
                const int page = id[0];
                id[0] = id[1];
                id[1] = id[2];
                id[2] = id[3];
                const uint32_t slot = q % SLOTS;
                uint64_t *full = &f8->full[kv][slot], *empty = &f8->empty[kv][slot];
                if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(empty, ((q / SLOTS) & 1) ^ 1))) store_scale();
                on = __all_sync(0xFFFFFFFFu, wait_phase(fd, empty, ((q / SLOTS) & 1) ^ 1) && !*reinterpret_cast<volatile int *>(&fd->dead));
                if (!on) break;
                ++q;
                const int key = key0 + k * kTcKeys + s * kRawTokens + lane;
                const int place = key - page_index(key) * psize;
                const bool good = (unsigned)page < (unsigned)a.c.n_pages;
                if (!good && page != kNoPage) report_error(a.stats, SV_ERR_INVALID_ARG, tab);
                const uint32_t scale = good ? my_scales[page * a.sc.page_b] : 127u;
                const uint32_t to = raw_base + slot * SLOT;
                bool rows = true;   // every lane has copies by rows on their way
                if (k < box_tiles) {
                    const int first = lane * a2.box_rows;   // of the lane's box
                    const int bpage = __shfl_sync(0xFFFFFFFFu, page, first & 31), bplace = __shfl_sync(0xFFFFFFFFu, place, first & 31);
                    const uint32_t split = SPLIT ? __ballot_sync(0xFFFFFFFFu, lane < boxes && bplace + 8 > psize) : 0;
                    if (elect_one()) mbar_expect_arrive_n(full, (kRawTokens - 8 * __popc(split)) * DP, 0);
                    __syncwarp();
                    // a bad page id lies outside the tensor and reads zeros
                    if (lane < boxes && !((split >> lane) & 1u)) box_load(to + first * DP, map, full, 0, h, bplace, bpage);
                    __syncwarp();
                    rows = false;
                    if (SPLIT && split) {
                        rows = true;
                        const int64_t off = good ? page * a.c.page_b + place * a.c.slot_b + h * a.c.head_b : -1;
#pragma unroll 1
                        for (int r0 = 0; r0 < kRawTokens; r0 += RPI) {
                            const int r = r0 + rsub;
                            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
                            const bool ok = o >= 0 && real;
                            if ((split >> (r >> 3)) & 1u) cp_async16(to + r * DP + ch * 16, src + (ok ? o + ch * 16 : 0), ok);
                        }
                    }
                } else {
                    const int64_t off = good ? page * a.c.page_b + place * a.c.slot_b + h * a.c.head_b : -1;
#pragma unroll 2
                    for (int r0 = 0; r0 < kRawTokens; r0 += RPI) {
                        const int r = r0 + rsub;
                        const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
                        const bool ok = o >= 0 && real;
                        cp_async16(to + r * DP + ch * 16, src + (ok ? o + ch * 16 : 0), ok);
                    }
                }
                if (rows) cp_async_arrive(full);
                else mbar_arrive(full);
                store_scale();   // of the slot before
                held = scale;
                held_slot = slot;
                holds = true;
            }
        }
    }
    store_scale();
    cp_async_commit();
    cp_async_wait<0>();   // no row is in flight when the block ends; boxes are when a wait gave up
    if (lane == 0) f8->next[kv] = q;
}

template <int DP, int SLOTS>
__device__ __forceinline__ void feed8_load(const AttendArgs &a, const TcArgs &a2, Feed *fd, Feed8 *f8, uint32_t raw_base, int kv, int lane) {
    if (a2.split) feed8_load_as<DP, SLOTS, true>(a, a2, fd, f8, raw_base, kv, lane);
    else feed8_load_as<DP, SLOTS, false>(a, a2, fd, f8, raw_base, kv, lane);
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

// One of the four widening warps: it also copies its quarter of the query tiles.  Stages at kv_base as feed_produce fills them; a
// stage is full when its two warps have arrived.
template <int DP, int STAGES, int QROWS, int SLOTS>
__device__ __forceinline__ void feed8_widen(const AttendArgs &a, Feed *fd, Feed8 *f8, uint32_t q_base, uint32_t kv_base, uint32_t raw_base, int wl,
                                            int lane) {
    constexpr int TILE = 128 * DP * 2, HALF = 128 * 128, SLOT = kRawTokens * DP;
    const int D = a.c.head_dim, kv = wl >> 1, sub = wl & 1;
    raw_base += kv * SLOTS * SLOT;
    // Eight lanes take two neighbouring tokens, four chunks each, of a token of eight different halves: neither the loads nor the
    // stores to the swizzled tile then meet in a bank.
    const int j = lane & 7, p = lane >> 3;
    const int row0 = DP == 128 ? (p >> 1) * 2 + (j >> 2) : p * 2 + (j >> 2);
    const int ch = DP == 128 ? (j & 3) + 4 * ((j >> 2) ^ (p & 1)) : j & 3;
    constexpr int PASS = DP == 128 ? 4 : 8;   // tokens of a pass
    const uint32_t from = row0 * DP + ch * 16, to_half = (ch >> 2) * HALF;
    uint32_t seq = kv, q_phases = 0, slots = sub;   // slots: the next of its ring
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
        for (int k = k0; k < k1 && on; ++k) {
            const uint32_t stage = seq % STAGES;
            on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &fd->kv_empty[stage], ((seq / STAGES) & 1) ^ 1));
            if (!on) break;
            seq += 2;
#pragma unroll 1
            for (int s = sub; s < 4 && on; s += 2, slots += 2) {
                const uint32_t slot = slots % SLOTS;
                on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &f8->full[kv][slot], (slots / SLOTS) & 1));
                if (!on) break;
                const uint32_t raw = raw_base + slot * SLOT + from;
                const uint32_t tile = kv_base + stage * TILE + s * (kRawTokens * 128) + to_half;
#pragma unroll 2
                for (int u = 0; u < kRawTokens / PASS; ++u) {
                    const int row = u * PASS + row0;
                    uint4 w;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                 : "r"(raw + u * (PASS * DP)));
                    const float f = *reinterpret_cast<volatile float *>(&f8->scale[kv][slot][row]);
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

inline bool cache_map8(CUtensorMap *map, char *base, const KvCache &c, int width, int box_rows) {
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.kv_heads, (cuuint64_t)c.page_size, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.head_b, (cuuint64_t)c.slot_b, (cuuint64_t)c.page_b};
    const cuuint32_t box[4] = {(cuuint32_t)width, 1, (cuuint32_t)box_rows, 1}, one[4] = {1, 1, 1, 1};
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// tc_args for codes: boxes of up to a slot's 32 tokens by whole heads.
inline TcArgs tc_args8(const KvCache &c, int width, uint32_t shape_s) {
    TcArgs t{};
    t.shape_s = shape_s;
    const int ps = c.page_size;
    t.page_shift = (ps & (ps - 1)) == 0 ? __builtin_ctz(ps) : -1;
    const int rows = ps % 32 == 0 ? 32 : ps % 16 == 0 ? 16 : ps >= 8 ? 8 : 0;
    t.split = rows == 8 && ps % 8 != 0;
    if (rows > 0) {
        t.box_rows = rows;
        if (encode_tiled() == nullptr || !cache_map8(&t.k, c.k, c, width, rows) || !cache_map8(&t.v, c.v, c, width, rows)) t.box_rows = 0;
    }
    return t;
}

}  // namespace sv
