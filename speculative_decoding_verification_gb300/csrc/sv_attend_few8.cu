// sv_attend_few8.cu — sv_kv_attend8 on the tensor cores for up to 32 packed rows a sequence and key head: bf16 queries, heads up to 128
// wide.  The products, groups and barriers are those of sv_attend_few.cu; what differs is how a cache in 8 bits comes to them.
//
// Codes are e4m3 numbers, which binary16 holds, so keys and values become binary16 tiles without their scales, one instruction a pair
// of codes.  Queries are binary16 too: a power of two brings the tile's largest to [2^14, 2^15), so what drops below 2^-24 is 2^-38 of it.  A
// row much smaller than another of its tile thus has scores off by up to 2^-39 of that other's largest: nothing, up to where
// float32 no longer resolves scores (2^22 and more, times log2(e)).  A power for each row, with a branch in the softmax for tiles that need
// them, took 511 us where this took 487 (both before weights had two parts).
//   scores    q' . code, times scale * 2^(key's exponent) * (the queries' power of two): a factor of the thread, whose token it is
//   weights   with E_j the exponent of token j's values, less the group's first token's,
//                 out = sum_j 2^(s_j) 2^(E_j) code_j / sum_j 2^(s_j) = sum_j w_j code_j / sum_j w_j 2^(-E_j),   w_j = 2^(s_j + E_j - M)
//             where M follows the largest s_j + E_j as a maximum does: weights are as exact as those of an unscaled cache whatever the
//             scales are.  A weight enters its product with the codes as two binary16 numbers, itself rounded and 2^11 times what that leaves,
//             rounded: within 2^-22 of it, or of the largest 2^-40 where that is more (half of binary16's last step, 2^-25, of 2^-11, beside 2^kLift).  One
//             number alone, off by up to 2^-11, took 462 us where this takes 491, and outputs would differ with how many rows a block has; without the 2^11
//             tokens beside one with nearly all the weight would have a number that is not much better.
//             An E_j below -40 is taken as -40 and the rest multiplies the weight, so that pages of zeros (whose scale is the least) count
//             in the sum.  E_j up to 64 leave every weight there that is within 2^-26 of its row's largest; above, the least may drop out.
// Keys are widened to tensor memory, from where the products take them, values to shared memory: its bandwidth (a tile of values is
// written, read, written wide and read by the products) would else be the bound.
// The walk's warp makes the query tiles, ahead of the products.  Blocks of eight columns without rows are left out of the softmax.
//
// A tile is 32 KB (heads of 128), 1,450 cycles of an SM's share of the measured copy bandwidth; long contexts take 2,120, and a piece's beginning
// and end some 7,000 on top.  What bounds it: latency, of the softmax's steps and of instruction fetches (the block's kinds of warps run
// more code than the caches next to them hold; the same instructions in another order are 3 to 20% slower or faster).  512 sequences x 6
// rows, 8 key heads of 128, 1,024 to 2,048 tokens: 491 us (the kernel of a bf16 cache: 525), 251 at the memory's rate.  64 sequences over
// 8,192 to 16,384 tokens: 360 us.  Heads of 64 halve the bytes and not the steps: 481 us, where the bf16 cache takes 366.
#include <float.h>

#define SV_WALK_PART static __host__ __device__ __noinline__

#include "sv_attend_feed8.cuh"
#include "sv_attend_few.cuh"

namespace sv {

namespace {

template <int DP>
struct Few8Shape {
    static constexpr int TILE = 128 * DP * 2;
    static constexpr int KST = DP == 128 ? 2 : 3, VST = DP == 128 ? 3 : 4;   // tiles of keys in tensor memory and of values in shared memory
    static constexpr int TOK = 64, SLOTS = 4;                     // tokens of a slot, slots of each ring of codes: two tiles
    static constexpr int HALF = 128 * 128;
    static constexpr int OFF_P = 2 * NR * DP * 2;                 // after two query tiles
    static constexpr int PBUF = 128 * 4 * NR;                     // a group's weights: 128 tokens x 32 rounded ones, 32 rests
    static constexpr int OFF_KV = OFF_P + 2 * PBUF;
    static constexpr int OFF_RAW = OFF_KV + VST * TILE;
    static constexpr int OFF_MISC = OFF_RAW + 2 * SLOTS * TOK * DP;
    // tensor memory: scores as in sv_attend_few.cu, a group's output (of the weights and of their rests), its 32 sums of each token's weights
    // twice, then keys
    static constexpr uint32_t COL_O = 128, COL_L = 256, COL_K = 384;
};
// Barriers of the tiles: kv_full, kv_empty [0, KST) are the keys', [KST, KST + VST) the values'.

struct Few8Shared : FewShared {
    Feed8 f8;
    float scale[2];                   // what the groups' outputs are in
    int unseen[2];                    // a row of the group has seen no token yet
};

// Weights are up to 2^(kGrow + kLift), where binary16 ends at 2^16: kGrow is how far a score may pass its maximum before that is taken anew.
constexpr float kLift = 4.0f, kGrow = 11.0f;
// Sums of weights are kept times 2^kSums: 2^(kSums - E_j) stays a normal number for every scale beside a first page of the least (E_j up to 167).
constexpr int kSums = 41;

// Two weights as pairs of binary16 numbers: each rounded, and 2^11 times what that leaves (at most half a step, 2^-11 of the weight, so no larger
// than that), rounded.
constexpr float kRestBack = 1.0f / 2048.0f;
__device__ __forceinline__ void weight_halves(f32x2 e, uint32_t &hi, uint32_t &lo) {
    float x, y, x11, y11;
    f2_unpack(e, x, y);
    f2_unpack(f2_mul(e, f2_pack(2048.0f, 2048.0f)), x11, y11);
    asm("{\n\t.reg .b16 a, b, m;\n\t.reg .f32 p, q;\n\t"
        "cvt.rn.f16x2.f32 %0, %3, %2;\n\t"
        "mov.b32 {a, b}, %0;\n\tmov.b16 m, 0xE800;\n\t"   // -2048
        "fma.rn.f32.f16 p, a, m, %4;\n\tfma.rn.f32.f16 q, b, m, %5;\n\t"
        "cvt.rn.f16x2.f32 %1, q, p;\n\t}"
        : "=&r"(hi), "=r"(lo)
        : "f"(x), "f"(y), "f"(x11), "f"(y11));
}

__device__ __forceinline__ float half_bits(uint16_t x) { return __half2float(*reinterpret_cast<const __half *>(&x)); }
__device__ __forceinline__ float weight_of(uint16_t hi, uint16_t lo) { return fmaf(half_bits(lo), kRestBack, half_bits(hi)); }

// scan_values for binary16 tiles of codes, where only NaN is not finite.
template <int DP>
__device__ __forceinline__ void scan_codes(uint32_t tile, int t, uint32_t *flags) {
    bool bad = false;
#pragma unroll
    for (int ch = 0; ch < DP / 8; ++ch) {
        const uint32_t at = tile + (ch >> 3) * (128 * 128) + t * 128 + (((ch & 7) ^ (t & 7)) << 4);
        uint32_t w[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
#pragma unroll
        for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7C00u) == 0x7C00u || (w[i] & 0x7C000000u) == 0x7C000000u;
    }
    if (bad) {
        const uint32_t zero[4] = {0, 0, 0, 0};
        for (int ch = 0; ch < DP / 8; ++ch) sts128(tile + (ch >> 3) * (128 * 128) + t * 128 + (((ch & 7) ^ (t & 7)) << 4), zero);
    }
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, bad);
    if ((t & 31) == 0) flags[t >> 5] = all;
    fence_async_smem();
}

// Adds to the group's output what the products left out: of each flagged token the values, NaN among them, times the weights that the product
// would have used, for the rows that see it.  t: the thread's head element.  Rare, and out of line for the sake of the loop that calls it (512 x 6 rows
// 475 us with it in line, 458 without, before weights had two parts).
template <int DP>
__device__ __noinline__ void add_unseen(const AttendArgs &a, const PieceInfo *pi, uint32_t *flags, int first, uint32_t colO, const char *weights, int t) {
#pragma unroll 1
    for (int j = 0; j < 128; ++j) {
        if (!((*reinterpret_cast<volatile uint32_t *>(&flags[j >> 5]) >> (j & 31)) & 1u)) continue;
        const int kk = first + j;
        const uint32_t see = rows_that_see(pi, kk, a.G, a.bt.n);
        if (kk >= pi->end) continue;   // flags mean nothing after a wait gave up
        const int64_t off = slot_offset(a.c, a.bt.page_table + pi->table * a.bt.table_pitch, kk);
        if (off < 0) continue;
        const float v = t < a.c.head_dim ? codes2(reinterpret_cast<const uint8_t *>(a.c.v + off + pi->h * a.c.head_b)[t]).x : 0.0f;
        const char *pj = weights + j * (4 * NR);
        uint32_t o[32];
        tmem_ld32(colO, o);
        tc_wait_ld();
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int at = (r & 7) * 2;
            const float w = weight_of(*reinterpret_cast<const uint16_t *>(pj + (((r >> 3) ^ (j & 7)) << 4) + at),
                                      *reinterpret_cast<const uint16_t *>(pj + ((((r >> 3) + 4) ^ (j & 7)) << 4) + at));
            if (((see >> r) & 1u) && r < pi->vr) o[r] = __float_as_uint(__uint_as_float(o[r]) + w * v);
        }
        tmem_st32(colO, o);
        tc_wait_st();
    }
}

// The same out of line, for the kernel of heads up to 64, where that leaves the loop's instructions better placed: 512 x 6 rows with heads of 48 and 64 482 and
// 481 us (556 in line), but of 80, 96 and 128 554 in the other kernel (491 to 494 in line).
template <int DP>
__device__ __noinline__ void scan_called(uint32_t tile, int t, uint32_t *flags) {
    scan_codes<DP>(tile, t, flags);
}

// The rest of token t's scale on its weights, as two numbers again.  Out of line as the above: heads of 64 481 us (493 in line).
__device__ __noinline__ void scale_weights(char *row, int t, uint32_t sees, float down, int vr) {
#pragma unroll 1
    for (int r = 0; r < vr; ++r) {
        uint16_t *at = reinterpret_cast<uint16_t *>(row + (r & 7) * 2 + (((r >> 3) ^ (t & 7)) << 4));
        uint16_t *rest = reinterpret_cast<uint16_t *>(row + (r & 7) * 2 + ((((r >> 3) + 4) ^ (t & 7)) << 4));
        const float w = (sees >> r) & 1u ? weight_of(*at, *rest) * down : 0.0f;   // NaN where it is seen
        *at = __half_as_ushort(__float2half_rn(w));
        *rest = __half_as_ushort(__float2half_rn((w - half_bits(*at)) * (1.0f / kRestBack)));
    }
}

// Reduction of x[0..7] over the warp's lanes: lane i gets that of x[i / 4].
template <class F>
__device__ __forceinline__ float reduce8(float (&x)[8], int lane, F f) {
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) {
        const bool up = lane & (4 * w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < w) {
                const float mine = up ? x[i + w] : x[i], other = up ? x[i] : x[i + w];
                x[i] = f(mine, __shfl_xor_sync(0xFFFFFFFFu, other, 4 * w));
            }
        }
    }
    float y = f(x[0], __shfl_xor_sync(0xFFFFFFFFu, x[0], 2));
    return f(y, __shfl_xor_sync(0xFFFFFFFFu, y, 1));
}

// Query tile of a piece, by one warp: rows of bf16 to binary16, all times one power of two.  Not finite numbers stay what they are and have no
// say in it.
template <int DP>
__device__ __forceinline__ void make_queries(const AttendArgs &a, PieceInfo *pi, uint32_t tile, int lane) {
    constexpr int CH = DP / 8, RPP = 32 / CH;   // chunks of a row, rows of a pass
    const int r0 = lane / CH, ch = lane % CH, vr = pi->vr, m0 = pi->m0;
    const bool real = ch * 8 < a.c.head_dim;
    // Copied to where they will be, all at once; a lane then finds the largest of its chunks, and rewrites them.
    const char *q = a.q + (int64_t)pi->r0 * a.q_row + (int64_t)pi->h * a.G * a.q_head + ch * 16;
    const int rows = ((vr + 7) & ~7) / RPP;   // passes: the softmax works on blocks of eight rows
    const uint32_t half = tile + (ch >> 3) * (NR * 128);
    auto place = [&](int pass) {
        const int r = pass * RPP + r0;
        return half + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
    };
    {
        // the lane's row of a pass, its head and place; the next pass's is RPP further
        const int i0 = (m0 + r0) / a.G, di = RPP / a.G, dg = RPP - di * a.G;
        int g = m0 + r0 - i0 * a.G;
        int64_t at = i0 * a.q_row + g * a.q_head;
        const int64_t step = di * a.q_row + dg * a.q_head, wrap = a.q_row - a.G * a.q_head;
#pragma unroll 1
        for (int pass = 0; pass < rows; ++pass) {
            const bool ok = pass * RPP + r0 < vr && real;
            cp_async16(place(pass), q + (ok ? at : -(int64_t)ch * 16), ok);
            g += dg;
            at += step;
            if (g >= a.G) {
                g -= a.G;
                at += wrap;
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
    }
    auto each = [&](auto use) {
#pragma unroll 2
        for (int pass = 0; pass < rows; ++pass) {
            uint4 w;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(place(pass)) : "memory");
            use(pass, w);
        }
    };
    // The largest finite number: bits of |x| rise as it does, so pairs are compared as whole numbers.  Infinities and NaN, above all others,
    // make it look again without them.
    uint32_t most2 = 0;
    each([&](int, uint4 w) {
        most2 = __vmaxu2(most2, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
    });
    uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(most2 & 0xFFFFu, most2 >> 16));
    if (most >= 0x7F80u) {
        most = 0;
        each([&](int, uint4 w) {
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = in[i] & 0x7FFFu, hi = (in[i] >> 16) & 0x7FFFu;
                most = max(most, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
            }
        });
        most = __reduce_max_sync(0xFFFFFFFFu, most);
    }
    const int up = most > 0 ? min(141 - (int)(most >> 7), 126) : 0;   // 2^up brings it to [2^14, 2^15)
    const float f = __uint_as_float((uint32_t)(127 + up) << 23);
    const f32x2 f2 = f2_pack(f, f);
    if (lane == 0) pi->q_back = __uint_as_float((uint32_t)(127 - up) << 23);
    each([&](int pass, uint4 w) {
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a0, a1;
            f2_unpack(f2_mul(f2_from_bf16x2(in[i]), f2), a0, a1);
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y[i]) : "f"(a1), "f"(a0));
        }
        sts128(place(pass), y);
    });
    fence_async_smem();
}

// One of the four widening warps: tokens 32 wl to 32 wl + 31 of each tile, half of a slot.  A lane takes one token's keys to tensor memory; of the
// values, eight lanes take two neighbouring tokens (WidenLane).
template <int DP>
__device__ __forceinline__ void widen_codes(Feed *fd, Feed8 *f8, uint32_t sbase, uint32_t tmem, int wl, int lane) {
    using S = Few8Shape<DP>;
    constexpr int SLOT = S::TOK * DP, PASS = WidenLane<DP>::PASS;
    const WidenLane<DP> me(lane);
    const uint32_t kraw = sbase + S::OFF_RAW + (wl & 1) * 32 * DP, vraw = kraw + S::SLOTS * SLOT + me.row0 * DP + me.ch * 16;
    const uint32_t vtile = sbase + S::OFF_KV + (me.ch >> 2) * S::HALF + wl * (32 * 128);
    const uint32_t kcol = tmem + S::COL_K + ((uint32_t)(wl * 32) << 16);
    static_assert(S::SLOTS == 4 && S::TOK == 64, "a slot goes to the same two warps each time");
    uint32_t n = 0;   // tiles
    bool on = true;
    for (int it = 0;; ++it) {
        const PieceInfo *pi = &fd->pd[it % kRing];
        if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1))) break;
        const int nk = pi->k1 - pi->k0;
        if (nk <= 0) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
        for (int k = 0; k < nk && on; ++k, ++n) {
            const uint32_t slot = (n & 1) * 2 + (wl >> 1), parity = (n >> 1) & 1;
            const uint32_t ks = n % S::KST, vs = n % S::VST;
            on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &f8->full[0][slot], parity) &&
                                             wait_phase(fd, &fd->kv_empty[ks], ((n / S::KST) & 1) ^ 1));
            if (!on) break;
            tc_fence_after();
#pragma unroll 1
            for (int half = 0; half < DP / 64; ++half) {   // 64 codes, four chunks
                uint32_t w[4][4], x[32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[c][0]), "=r"(w[c][1]), "=r"(w[c][2]), "=r"(w[c][3])
                                 : "r"(kraw + slot * SLOT + raw_place<DP, true>(lane, half * 4 + c)));
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) codes4_f16(w[c][j], x[c * 8 + 2 * j], x[c * 8 + 2 * j + 1]);
                tmem_st32(kcol + ks * (DP / 2) + half * 32, x);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&f8->empty[0][slot]);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&fd->kv_full[ks]);

            on = __all_sync(0xFFFFFFFFu, wait_phase(fd, &f8->full[1][slot], parity) &&
                                             wait_phase(fd, &fd->kv_empty[S::KST + vs], ((n / S::VST) & 1) ^ 1));
            if (!on) break;
#pragma unroll 1
            for (int u = 0; u < 32 / PASS; u += 4) {
                uint32_t w[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                                 : "r"(vraw + slot * SLOT + (u + i) * (PASS * DP)));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = (u + i) * PASS + me.row0, c = 2 * (me.ch & 3);
                    uint32_t lo[4], hi[4];
                    codes4_f16(w[i][0], lo[0], lo[1]);
                    codes4_f16(w[i][1], lo[2], lo[3]);
                    codes4_f16(w[i][2], hi[0], hi[1]);
                    codes4_f16(w[i][3], hi[2], hi[3]);
                    sts128(vtile + vs * S::TILE + row * 128 + ((c ^ (row & 7)) << 4), lo);
                    sts128(vtile + vs * S::TILE + row * 128 + (((c + 1) ^ (row & 7)) << 4), hi);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&f8->empty[1][slot]);
                mbar_arrive(&fd->kv_full[S::KST + vs]);
            }
        }
    }
}

// The warp that issues the products, run by the whole warp with uniform values: S^T = K Q^T of a tile, keys from tensor memory, and two tiles
// behind O^T += V^T P^T, so that a group finds its next scores made when it has written its weights.  One loop with one copy of each:
// the block's kinds of warps share the instruction cache, and with the weighted sum at five places, and loops like this laid out in full
// elsewhere, five in six cycles of the running warps went to missing instructions.
template <int DP>
__device__ __forceinline__ void issue_products(Feed *fd, FewShared *ms, uint32_t shape_s, uint32_t shape_o, uint32_t sbase, uint32_t tmem, int lane) {
    using S = Few8Shape<DP>;
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    uint32_t n = 0, tiles0 = 0, tiles1 = 0;   // tiles in all and of the groups
    int rests = 0;                            // as in the softmax
    // Tiles [weighed, n), three at most, have scores and no weighted sum yet: a bit each, the oldest lowest, for their groups and for the
    // parities of their places in them.
    uint32_t weighed = 0, groups = 0, parities = 0;
    int it = -1, i = 0, nk = 0, first = 0;    // piece, tile of it and their number, first group
    bool ends = false;
    for (;;) {
        // What comes next, a piece or a tile, waits for two barriers.  While they are not complete the weighted sums go ahead.
        const bool piece = i == nk;
        const int gr = first ^ (i & 1);   // of the tile
        const int next = piece ? it + 1 : it;
        uint64_t *b0 = piece ? &fd->pd_full[next % kRing] : &fd->kv_full[n % S::KST], *b1 = !piece && i == 0 ? &fd->q_full[it & 1] : b0;
        const uint32_t p0 = piece ? next / kRing & 1 : n / S::KST & 1, p1 = !piece && i == 0 ? it >> 1 & 1 : p0;
#pragma unroll 1
        while (weighed < n && (sum_is_due(n - weighed, groups, piece ? -1 : gr) || ends || !__all_sync(0xFFFFFFFFu, mbar_test_wait(b0, p0) && mbar_test_wait(b1, p1)))) {
            const uint32_t stage = weighed % S::VST, of = groups & 1;
            wait_phase(fd, &fd->kv_full[S::KST + stage], (weighed / S::VST) & 1);
            wait_phase(fd, &ms->p_full[of], parities & 1);
            __syncwarp();
            tc_fence_after();
            const uint64_t v = smem_operand(sbase + S::OFF_KV + stage * S::TILE, DP == 128 ? S::HALF : 0, 1024);
            const uint64_t p = smem_operand(sbase + S::OFF_P + of * S::PBUF, 0, 1024);
            const uint32_t o = tm + S::COL_O + of * (2 * NR);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) mma_ss(o, v + kk * (2048 >> 4), p + kk * (2048 >> 4), shape_o, 1u);
                mma_commit(&fd->kv_empty[S::KST + stage]);
                mma_commit(&ms->p_done[of]);
            }
            __syncwarp();
            ++weighed;
            groups >>= 1;
            parities >>= 1;
        }
        if (ends) break;
        if (piece) {
            ++it;
            i = 0;
            const bool more = __all_sync(0xFFFFFFFFu, wait_phase<true>(fd, b0, p0));
            const PieceInfo *pi = &fd->pd[it % kRing];
            nk = more ? __shfl_sync(0xFFFFFFFFu, pi->k1 - pi->k0, 0) : 0;
            if (nk <= 0) {
                nk = 0;
                ends = true;
                continue;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
            if (nk == 1) rests ^= 1;
            first = __shfl_sync(0xFFFFFFFFu, nk == 1 ? rests ^ 1 : 0, 0);   // uniform for the compiler too
            continue;
        }
        wait_phase(fd, b0, p0);
        wait_phase(fd, b1, p1);
        __syncwarp();
        tc_fence_after();
        const uint32_t stage = n % S::KST, u = gr ? tiles1 : tiles0;
        const uint32_t sc = tm + (gr * 2 + (u & 1)) * 32, kt = tm + S::COL_K + stage * (DP / 2);
        const uint64_t q = smem_operand(sbase + (it & 1) * (NR * DP * 2), 16, 1024);
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                const uint32_t qa = ((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4;
                mma_ts(sc, kt + kk * 8, q + qa, shape_s, kk > 0);
            }
            mma_commit(&ms->s_full[gr][u & 1]);
            mma_commit(&fd->kv_empty[stage]);
            if (i == nk - 1) mma_commit(&fd->q_empty[it & 1]);
        }
        __syncwarp();
        groups |= gr << (n - weighed);
        parities |= (u & 1) << (n - weighed);
        if (gr) ++tiles1;
        else ++tiles0;
        ++n;
        ++i;
    }
    if (elect_one()) mma_commit(&ms->done);
    wait_phase<true>(fd, &ms->done, 0);   // the products end by themselves
    __syncwarp();
}

template <int DP>
__global__ void __launch_bounds__(kTcThreads, 1) k_attend_few8(const __grid_constant__ AttendArgs a, const __grid_constant__ TcArgs a2) {
    using S = Few8Shape<DP>;
    extern __shared__ __align__(1024) char smem[];
    Few8Shared *ms = reinterpret_cast<Few8Shared *>(smem + S::OFF_MISC);
    Feed *fd = &ms->fd;
    Feed8 *f8 = &ms->f8;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

    if (smem_addr(smem) & 1023) {   // the swizzle goes by address bits
        if (tid == 0) report_error(a.stats, SV_ERR_CUDA, -1);
        return;
    }
    if (tid == 0) {
        feed_init(fd, a, kFewReaders + 2, 4, 1);
        feed8_init(f8, S::SLOTS, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms->s_full[i][0], 1);
            mbar_init(&ms->s_full[i][1], 1);
            mbar_init(&ms->p_full[i], 4);
            mbar_init(&ms->p_done[i], 1);
        }
        mbar_init(&ms->done, 1);
        for (int i = 0; i < NR; ++i) ms->zero[i] = 0.0f;
        fence_barrier_init();
    }
    if (warp == 12) tmem_alloc(&fd->tmem, 512);
    tc_fence_before();
    walk_start<kTcThreads>(a, &ms->walk, ms->warp_sum);   // has block-wide barriers
    pdl_trigger();
    tc_fence_after();
    const uint32_t tmem = fd->tmem;
    const uint32_t sbase = smem_addr(smem);

    if (warp < 8) {
        // ---------------------------------------------------------------- softmax
        const int gr = warp >> 2, wl = warp & 3, t = wl * 32 + lane;   // group, warp of it, token of the tile (head element at the end)
        const uint32_t base = tmem + ((uint32_t)(wl * 32) << 16);
        const uint32_t colO = base + S::COL_O + gr * (2 * NR), colL = base + S::COL_L + gr * (2 * NR);
        const uint32_t prow = sbase + S::OFF_P + gr * S::PBUF + t * (4 * NR);     // this token's weights; chunk q at q ^ (t & 7)
        uint32_t u = 0;   // tiles this group has worked on
        int rests = 0;    // the group that left the last piece of one tile to the other
        auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + gr) : "memory"); };
        auto page_of = [&](const PieceInfo *p, int k, int token) {
            const int key = min(p->key0 + k * kTcKeys + token, p->end - 1);
            return a.bt.page_table[p->table * a.bt.table_pitch + (a2.page_shift >= 0 ? key >> a2.page_shift : key / a.c.page_size)];
        };
        for (int it = 0;; ++it) {
            const PieceInfo *pi = &fd->pd[it % kRing];
            if (!wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1)) break;
            __syncwarp();
            const int k0 = pi->k0, k1 = pi->k1;
            if (k0 >= k1) break;
            const bool solo = k1 - k0 == 1;   // one group works on it, the other goes on to the next piece
            if (solo) {
                rests ^= 1;
                if (rests == gr) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
                    continue;
                }
            }
            const int key0 = pi->key0, ctx = pi->ctx, vr = pi->vr, used = (vr + 7) >> 3;   // used: blocks of eight rows
            // This thread's token's scales: pages are looked up two tiles of the group ahead, scales one.  A warp stops at the first use
            // of a load that is still on its way, so what is loaded ahead is not looked at, not even to leave it out: a token past the
            // unit's last takes the last one's, and a bad page is page 0's until its scales are used.
            const uint8_t *ks = a.sc.k + pi->h * a.sc.head_b, *vs8 = a.sc.v + pi->h * a.sc.head_b;
            auto good = [&](int page) { return (unsigned)page < (unsigned)a.c.n_pages; };
            auto byte_of = [&](const uint8_t *scales, int page) -> uint32_t { return scales[(good(page) ? page : 0) * a.sc.page_b]; };
            {
                uint32_t zero[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) zero[j] = 0;
                tmem_st32(colO, zero);
                tmem_st32(colO + NR, zero);
                tmem_st32(colL, zero);
                tc_wait_st();
            }
            float *shift = ms->shift[gr], *alpha = ms->alpha[gr];
            bool unseen = true, flip = false;   // flip: the sums are in the upper half of their columns
            const int begin = solo ? k0 : k0 + gr;
            float cq = 0.0f;   // what scores are multiplied by, but for the key's scale
            int page = page_of(pi, begin, t), page_next = page_of(pi, begin + 2, t);
            const int page0 = page_of(pi, begin, 0);
            uint32_t kb_next = byte_of(ks, page), vb_next = byte_of(vs8, page);
            const uint32_t v0 = byte_of(vs8, page0);
            for (int k = begin; k < k1; k += 2, ++u) {
                const int buf = u & 1;
                const uint32_t colS = base + (gr * 2 + buf) * 32;
                wait_phase(fd, &ms->s_full[gr][buf], (u >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                const uint32_t kb = good(page) ? kb_next : 127u, vb = good(page) ? vb_next : 127u;
                page = page_next;
                kb_next = byte_of(ks, page);
                vb_next = byte_of(vs8, page);
                page_next = page_of(pi, k + 4, t);
                const int e0 = min(max((int)v0, 127 - 40), 127 + 40);   // byte that the values' scales are taken from
                if (k == begin) cq = a.scale_log2 * *reinterpret_cast<const volatile float *>(&pi->q_back);
                const float cs = fminf(cq, FLT_MAX) * scale_of(kb);
                const f32x2 c2 = f2_pack(cs == INFINITY ? FLT_MAX : cs, cs == INFINITY ? FLT_MAX : cs);
                const int ev = (int)vb - e0, up = vb == 255 ? 0 : max(ev, -40);
                const float lift = (float)up;
                const float down = vb == 255 ? NAN : ev < -40 ? pow2i(ev + 40) : 1.0f;   // the rest of the scale
                const f32x2 lift2 = f2_pack(lift, lift), back = f2_pack(pow2i(kSums - up), pow2i(kSums - up));
                const bool masked = key0 + (k + 1) * kTcKeys > ctx;
                const uint32_t sees = masked ? rows_that_see(pi, key0 + k * kTcKeys + t, a.G, a.bt.n) : 0xFFFFFFFFu;
                // the group's previous product has read the weights and written the output
                if (u > 0) wait_phase(fd, &ms->p_done[gr], (u - 1) & 1);
                __syncwarp();
                tc_fence_after();
                // Everything goes by blocks of eight rows, in rolled loops that read the scores anew: what the softmax would hold
                // unrolled in registers costs more in instruction fetches (736 us for 512 x 6 rows over 1-2k tokens, where this took 487).
                auto scores = [&](int q, const float *less, float (&x)[8]) {
                    uint32_t raw[8];
                    tmem_ld8(colS + 8 * q, raw);
                    tc_wait_ld();
#pragma unroll
                    for (int r = 0; r < 8; r += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(less + 8 * q + r);
                        f2_unpack(f2_fma(f2_from_u32x2(raw[r], raw[r + 1]), c2, f2_add(f2_pack(m.x, m.y), lift2)), x[r], x[r + 1]);
                        f2_unpack(f2_fma(f2_from_u32x2(raw[r + 2], raw[r + 3]), c2, f2_add(f2_pack(m.z, m.w), lift2)), x[r + 2], x[r + 3]);
                    }
                    if (masked) {
                        const uint32_t bits = sees >> (8 * q);
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            if (!((bits >> r) & 1u)) x[r] = -INFINITY;
                    }
                };
                // Weights are made from the maxima as they are.  Where a score passes its row's by 2^kGrow the group takes the maxima anew and
                // makes the tile's weights again, as it does first of all until every row has seen a token.  The sums before the
                // tile stay where they were: the tile's go to the other half.
                const uint32_t sums = colL + (flip ? NR : 0), sums_to = colL + (flip ? 0 : NR);
#pragma unroll 1
                for (uint32_t grow = unseen;; grow = 1) {
                    if (grow) {
#pragma unroll 1
                        for (int q = 0; q < used; ++q) {
                            float x[8];
                            scores(q, ms->zero, x);
                            const float top = reduce8(x, lane, [](float p, float q) { return fmaxf(p, q); });
                            if ((lane & 3) == 0) ms->top[gr][wl][8 * q + (lane >> 2)] = top;
                        }
                        group_sync();
                        if (wl == 0) {
                            const float old = k > begin ? kLift - shift[lane] : kNoMax;
                            const float now = fmaxf(fmaxf(fmaxf(ms->top[gr][0][lane], ms->top[gr][1][lane]), old),
                                                    fmaxf(ms->top[gr][2][lane], ms->top[gr][3][lane]));
                            alpha[lane] = ex2_fast(old - now);
                            shift[lane] = kLift - now;
                            const bool none = __any_sync(0xFFFFFFFFu, lane < vr && now == kNoMax);
                            if (lane == 0) ms->unseen[gr] = none;
                        }
                        group_sync();
                        unseen = *reinterpret_cast<volatile int *>(&ms->unseen[gr]);
                        if (k > begin) {
#pragma unroll 1
                            for (int q = 0; q < used; ++q) {
                                uint32_t o[8], o2[8], l[8];
                                tmem_ld8(colO + 8 * q, o);
                                tmem_ld8(colO + NR + 8 * q, o2);
                                tmem_ld8(sums + 8 * q, l);
                                tc_wait_ld();
#pragma unroll
                                for (int r = 0; r < 8; ++r) {
                                    const float f = alpha[8 * q + r];
                                    o[r] = __float_as_uint(__uint_as_float(o[r]) * f);
                                    o2[r] = __float_as_uint(__uint_as_float(o2[r]) * f);
                                    l[r] = __float_as_uint(__uint_as_float(l[r]) * f);
                                }
                                tmem_st8(colO + 8 * q, o);
                                tmem_st8(colO + NR + 8 * q, o2);
                                tmem_st8(sums + 8 * q, l);
                            }
                            tc_wait_st();
                        }
                    }
                    float over = -INFINITY;
#pragma unroll 1
                    for (int q = 0; q < used; ++q) {   // eight rows' weights, a 16-byte chunk
                        float x[8];
                        uint32_t l[8], w[4], rest[4];
                        tmem_ld8(sums + 8 * q, l);
                        scores(q, shift, x);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            over = fmaxf(over, fmaxf(x[2 * j], x[2 * j + 1]));
                            const f32x2 e = f2_ex2(f2_pack(x[2 * j], x[2 * j + 1]));
                            float y, z;
                            f2_unpack(f2_fma(e, back, f2_from_u32x2(l[2 * j], l[2 * j + 1])), y, z);
                            l[2 * j] = __float_as_uint(y);
                            l[2 * j + 1] = __float_as_uint(z);
                            weight_halves(e, w[j], rest[j]);
                        }
                        tmem_st8(sums_to + 8 * q, l);
                        sts128(prow + ((q ^ (t & 7)) << 4), w);
                        sts128(prow + (((q + 4) ^ (t & 7)) << 4), rest);
                    }
                    if (grow) break;
                    uint32_t again;
                    asm volatile(
                        "{\n\t.reg .pred p, q;\n\tsetp.gt.f32 p, %1, %3;\n\t"
                        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                        : "=r"(again)
                        : "f"(over), "r"(1 + gr), "f"(kGrow + kLift)
                        : "memory");
                    if (!again) break;
                    tc_wait_st();
                }
                flip = !flip;
                if (down != 1.0f) scale_weights(smem + S::OFF_P + gr * S::PBUF + t * (4 * NR), t, sees, down, vr);
                if (masked) {
                    // Codes that are NaN are replaced by zeros; they are added here for the rows that see them, with the weights that the
                    // product would have used.
                    const uint32_t n = pi->seq / 2 + (k - k0), stage = n % S::VST;
                    wait_phase(fd, &fd->kv_full[S::KST + stage], (n / S::VST) & 1);
                    __syncwarp();
                    if constexpr (DP == 64) scan_called<DP>(sbase + S::OFF_KV + stage * S::TILE, t, fd->vflag[stage]);
                    else scan_codes<DP>(sbase + S::OFF_KV + stage * S::TILE, t, fd->vflag[stage]);
                    group_sync();   // the flags and every token's weights are written
                    uint32_t any = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) any |= *reinterpret_cast<volatile uint32_t *>(&fd->vflag[stage][q]);
                    if (any) {
                        add_unseen<DP>(a, pi, fd->vflag[stage], key0 + k * kTcKeys, colO, smem + S::OFF_P + gr * S::PBUF, t);
                    }
                }
                tc_wait_st();
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms->p_full[gr]);
            }
            // ---- the piece's end: thread t has head element t
            const int D = a.c.head_dim, qh0 = pi->h * a.G, r0 = pi->r0;
            const bool whole = pi->whole;
            const int ga = solo ? gr : 0;                      // the group that works on it, or the first of the two
            const int bar = solo ? 1 + gr : 3, threads = solo ? 128 : 256;
            auto end_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory"); };
            const size_t slot = (size_t)pi->slot;
#pragma unroll 1
            for (int q = 0; q < used; ++q) {
                uint32_t l[8];
                float x[8];
                tmem_ld8(colL + (flip ? NR : 0) + 8 * q, l);
                tc_wait_ld();
#pragma unroll
                for (int r = 0; r < 8; ++r) x[r] = __uint_as_float(l[r]);
                const float sum = reduce8(x, lane, [](float p, float q) { return p + q; });
                if ((lane & 3) == 0) ms->top[gr][wl][8 * q + (lane >> 2)] = sum;
            }
            if (t == 0) ms->scale[gr] = scale_of(min(max((int)v0, 127 - 40), 127 + 40) + kSums);
            __syncwarp();
            if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
            end_sync();
            if (warp == ga * 4) {
                auto sum_of = [&](int g) { return (ms->top[g][0][lane] + ms->top[g][1][lane]) + (ms->top[g][2][lane] + ms->top[g][3][lane]); };
                float m = -ms->shift[ga][lane] - kSums, f0 = 1.0f, f1 = 0.0f, all = sum_of(ga);
                if (!solo) {
                    const float top0 = m, top1 = -ms->shift[1][lane] - kSums;
                    m = fmaxf(top0, top1);
                    f0 = ex2_fast(top0 - m);
                    f1 = ex2_fast(top1 - m);
                    all = all * f0 + sum_of(1) * f1;
                }
                const float inv = whole ? (all > 0.0f || all != all ? 1.0f / all : 0.0f) : 1.0f;
                ms->alpha[ga][lane] = f0 * inv * ms->scale[ga];
                if (!solo) ms->alpha[1][lane] = f1 * inv * ms->scale[1];
                if (lane < vr) {
                    if (!whole) {
                        a.part_ml[slot + lane] = make_float2(m, all);
                    } else if (a.lse) {
                        const int i = lane / a.G, g = lane - i * a.G;
                        a.lse[(size_t)(r0 + i) * a.q_heads + qh0 + g] = all == 0.0f ? -INFINITY : (m + log2f(all)) / kLog2e;
                    }
                }
            } else if (warp == (solo ? ga * 4 + 1 : 4)) {   // meanwhile
                const int i = lane / a.G, g = lane - i * a.G;
                ms->to[ga][lane] = (int64_t)(r0 + i) * a.o_row + (int64_t)(qh0 + g) * a.o_head;
            }
            wait_phase(fd, &ms->p_done[gr], (u - 1) & 1);
            end_sync();
            tc_fence_after();
            // Four rows at a time, the groups taking turns, as in sv_attend_few.cu.
#pragma unroll 1
            for (int rb = solo ? 0 : gr * 4; rb < vr; rb += solo ? 4 : 8) {
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
                for (int g = ga; g < (solo ? ga + 1 : 2); ++g) {
                    uint32_t o[4], o2[4];   // the products with the weights and with their rests
                    tmem_ld4(base + S::COL_O + g * (2 * NR) + rb, o);
                    tmem_ld4(base + S::COL_O + g * (2 * NR) + NR + rb, o2);
                    tc_wait_ld();
                    const float4 f = *reinterpret_cast<const float4 *>(ms->alpha[g] + rb);
                    y[0] = fmaf(fmaf(__uint_as_float(o2[0]), kRestBack, __uint_as_float(o[0])), f.x, y[0]);
                    y[1] = fmaf(fmaf(__uint_as_float(o2[1]), kRestBack, __uint_as_float(o[1])), f.y, y[1]);
                    y[2] = fmaf(fmaf(__uint_as_float(o2[2]), kRestBack, __uint_as_float(o[2])), f.z, y[2]);
                    y[3] = fmaf(fmaf(__uint_as_float(o2[3]), kRestBack, __uint_as_float(o[3])), f.w, y[3]);
                }
                if (t < D) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (rb + r >= vr) continue;
                        if (whole) store_elem<2>(a.out + ms->to[ga][rb + r] + t * 2, y[r]);
                        else a.part[(slot + rb + r) * D + t] = y[r];
                    }
                }
            }
            tc_fence_before();
            end_sync();   // outputs, sums and maxima may be written again
        }
    } else if (warp < 12) {
        widen_codes<DP>(fd, f8, sbase, tmem, warp - 8, lane);
    } else {
        if (warp == 12) {   // V transposed times the weights
            issue_products<DP>(fd, ms, a2.shape_s, mma_shape_f16(2 * NR, true, true, false, false), sbase, tmem, lane);
        } else if (warp == 13) {
            feed_walk(a, a2, fd, ms->walk, lane, [&](int it) {
                if (__all_sync(0xFFFFFFFFu, wait_phase(fd, &fd->q_empty[it & 1], ((it >> 1) & 1) ^ 1))) {
                    make_queries<DP>(a, &fd->pd[it % kRing], sbase + (it & 1) * (NR * DP * 2), lane);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&fd->q_full[it & 1]);
                }
            });
        } else {
            feed8_load<DP, S::TOK, S::SLOTS, false, true, true>(a, a2, fd, f8, sbase + S::OFF_RAW + (warp - 14) * (S::SLOTS * S::TOK * DP), warp - 14, lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && fd->dead) feed8_drain<S::SLOTS>(fd, f8, a.stats);
    if (warp == 12) tmem_free(tmem, 512);
    pdl_wait();   // launched beside the prefixes' kernel: done only when that is, for the join waits for this one
}

template <int DP>
cudaError_t run_few8(AttendArgs &a, bool negate, cudaStream_t stream) {
    constexpr size_t bytes = Few8Shape<DP>::OFF_MISC + sizeof(Few8Shared);
    static_assert(bytes <= 232448, "shared memory of a block");
    if (prepare_kernel((const void *)k_attend_few8<DP>, kTcThreads, bytes) < 1) return cudaErrorInvalidConfiguration;
    const TcArgs t = tc_args8(a.c, DP, true, mma_shape_f16(NR, false, false, false, negate));
    // After the prefixes' kernel of the same call, blocks start as that one's end: they need nothing of it.
    if (a.geo.s0 > 0) return launch_pdl(k_attend_few8<DP>, dim3(a.geo.blocks), dim3(kTcThreads), bytes, stream, a, t);
    k_attend_few8<DP><<<a.geo.blocks, kTcThreads, bytes, stream>>>(a, t);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_few8(AttendArgs &a, cudaStream_t stream) {
    static_assert(kTilesFew.TM == NR && kTilesFew.TK == kTcKeys, "the cutting's tiles are the kernel's");
    a.geo.set(kTilesFew);
    AttendArgs t = a;
    // The maximum is taken after the scale; a negative scale negates the queries in the product, and zero stays zero.
    const bool negate = a.scale_log2 < 0.0f;
    t.scale_log2 = fabsf(a.scale_log2);
    return a.c.head_dim <= 64 ? run_few8<64>(t, negate, stream) : run_few8<128>(t, negate, stream);
}

}  // namespace sv
