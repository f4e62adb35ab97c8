// sv_attend_tall.cu — sv_kv_attend on the tensor cores for any number of rows: bf16, heads up to 128 wide.
//
// A persistent block of 16 warps walks its range of (unit, key tile)s; units are 256 packed rows, key tiles 128 tokens.
//   warps 0-3, 4-7   softmax of two streams: a thread owns one row of 128 scores in tensor memory
//   warps 8-11       producers: gather keys, values and queries from their pages into swizzled shared memory
//   warp 12          issues the matrix products
//   warp 13          walks the range and describes the pieces to the others, a few ahead
// Streams.  A piece of more than 128 rows is two row tiles that share each key tile, one a stream.  A piece of up to 128 rows
// is one row tile whose even key tiles go to one stream and odd ones to the other, each with its own maximum, sum and
// output, added at the piece's end.  Either way one stream's products run while the other's softmax does.
// Tensor memory (512 columns): scores 2 x 128, the weights over the scores they came from, outputs 2 x 128.
// Weights.  A weight enters the product with V as two bf16 parts, its upper bits and the rounded rest (16 bits in all): one
// part alone is off by 2^-8, as much as the rounding of the output.
//
// What bounds it: a stream's softmax (1,600 cycles a tile of 128 x 128) and its products (1,536: 8 for the scores, 16 for the weighted
// sum, 64 cycles each) follow one another; the two streams together take 4,060 cycles for a pair of tiles, against 3,077 for the
// products alone.  64 x 6 rows of 32 heads over a prefix of 32,768 tokens: 213 us, 62% of tensor cycles.  One warp issues for both
// streams: with a warp a stream their products interleave and each ends later (355 us for the call against 300).
#include <float.h>

#include "sv_attend_feed8.cuh"

namespace sv {

namespace {

constexpr int kTallRows = 256;
constexpr int kTallReaders = 13;      // warps that read a piece description
constexpr uint32_t kColS = 0, kColO = 256;

// C8: the cache is held in 8 bits.  Codes become the bf16 tiles of before (sv_attend_feed8.cuh), so results are those of a bf16 cache of the same values
// to the bit; what they cost is the widening, four warps' five instructions a pair of codes, once for each row tile: 2 sequences x
// 1,300 rows over 3,000 tokens 298 us (241 over bf16), the prompt above 316 us for the whole call (284), 16 trees of 57 rows 70 us (60).
template <int DP, bool C8>
struct TallShape {
    static constexpr int TILE = 128 * DP * 2;              // bytes of 128 rows
    static constexpr int STAGES = DP == 64 ? 8 : C8 ? 4 : 5;
    static constexpr int SLOTS = DP == 64 ? 8 : 3;         // of each ring of codes
    static constexpr int HALF = 128 * 128;                 // bytes of 128 rows of 64 elements
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_RAW = OFF_KV + STAGES * TILE;
    static constexpr int OFF_MISC = OFF_RAW + (C8 ? 2 * SLOTS * kRawTokens * DP : 0);
};

struct TallShared {
    Feed fd;
    uint64_t s_full[2], p_half[2], p_full[2], o_full[2], done;   // p_half: the first 64 tokens' weights
    union {
        struct {
            Walk walk;                // read before the first piece is described
            long long warp_sum[kTcThreads / 32];
        };
        float2 ml[2][128];            // maxima and sums exchanged by the streams
    };
};

struct TallShared8 : TallShared {
    Feed8 f8;
};

// Bits of the 128 tokens first .. first + 127 that a row of a tree sees, from its ancestor bits.
__device__ __forceinline__ uint32_t anc_at(const uint32_t (&anc)[5], int k) {
    if (k < 0) return 0xFFFFFFFFu;   // cached tokens
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i)
        if (i == k) w = anc[i];
    return w;
}

template <int DP, bool C8>
__global__ void __launch_bounds__(kTcThreads, 1) k_attend_tall(const __grid_constant__ AttendArgs a, const __grid_constant__ TcArgs a2) {
    using S = TallShape<DP, C8>;
    extern __shared__ __align__(1024) char smem[];
    TallShared *ms = reinterpret_cast<TallShared *>(smem + S::OFF_MISC);
    Feed *fd = &ms->fd;
    Feed8 *f8 = C8 ? &static_cast<TallShared8 *>(ms)->f8 : nullptr;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

    if (smem_addr(smem) & 1023) {   // the swizzle goes by address bits
        if (tid == 0) report_error(a.stats, SV_ERR_CUDA, -1);
        return;
    }
    if (tid == 0) {
        feed_init(fd, a, C8 ? kTallReaders + 2 : kTallReaders, C8 ? 2 : 64, 128);
        if (C8) feed8_init(f8, S::SLOTS, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms->s_full[i], 1);
            mbar_init(&ms->p_half[i], 4);
            mbar_init(&ms->p_full[i], 4);
            mbar_init(&ms->o_full[i], 1);
        }
        mbar_init(&ms->done, 1);
        fence_barrier_init();
    }
    if (warp == 12) tmem_alloc(&fd->tmem, 512);
    tc_fence_before();
    walk_start<kTcThreads>(a, &ms->walk, ms->warp_sum);   // has block-wide barriers
    pdl_trigger();
    tc_fence_after();
    const uint32_t tmem = fd->tmem;

    if (warp < 8) {
        regs_inc<kRegsSoftmax>();
        // ---------------------------------------------------------------- softmax
        const int st = warp >> 2;                               // stream
        const int wl = warp & 3, row = wl * 32 + lane;          // tensor-memory lane
        const uint32_t base = tmem + ((uint32_t)(wl * 32) << 16);
        const uint32_t colS = base + kColS + st * 128, colO = base + kColO + st * 128;
        uint32_t s_phase = 0, o_phases = 0, seq = 0;   // o_phases: a bit a stream
        const float c = a.scale_log2;
        for (int it = 0;; ++it) {
            PieceInfo *pi = &fd->pd[it % kRing];
            if (!wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1)) break;
            const int k0 = pi->k0, k1 = pi->k1;
            if (k0 >= k1) break;
            __syncwarp();
            const int vr = pi->vr, key0 = pi->key0, ctx = pi->ctx, own = pi->own, tree = pi->tree, end = pi->end;
            const bool two = vr > 128;
            const int m = two ? st * 128 + row : row;           // row of the unit
            const int i = (pi->m0 + m) / a.G;                   // row of the segment
            const bool active = (two ? st * 128 : 0) + wl * 32 < vr;   // the warp has rows
            uint32_t anc[5] = {0, 0, 0, 0, 0};
            if (tree && m < vr) {
                for (int j = i;;) {
#pragma unroll
                    for (int k = 0; k < 5; ++k)
                        if ((j >> 5) == k) anc[k] |= 1u << (j & 31);
                    if (j == 0) break;
                    const int p = pi->par[j - 1];
                    if (p == 255) break;
                    j = p;
                }
            }
            const int lim = !own ? end : tree ? ctx : min(ctx + i + 1, end);
            if (active) {
                uint32_t zero[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) zero[j] = 0;
#pragma unroll
                for (int j = 0; j < DP; j += 32) tmem_st32(colO + j, zero);
            }
            float m_used = -INFINITY, l = 0.0f;
            const int step = two ? 1 : 2, begin = two ? k0 : k0 + st;
            for (int k = begin; k < k1; k += step) {
                wait_phase(fd, &ms->s_full[st], s_phase);
                s_phase ^= 1;
                __syncwarp();
                const int first = key0 + k * kTcKeys;
                const bool masked = own ? first + kTcKeys > ctx : first + kTcKeys > end;
                // Tokens that some row does not see: the stream's threads (the first stream's, where both share the tile, whose
                // products come first) clear values that are not finite.
                const uint32_t vs = seq + 2 * (k - k0) + 1, vstage = vs % S::STAGES;
                if (own && masked) {
                    if (!two || st == 0) {
                        wait_phase(fd, &fd->kv_full[vstage], (vs / S::STAGES) & 1);
                        __syncwarp();
                        scan_values<DP>(smem_addr(smem) + S::OFF_KV + vstage * S::TILE, row, fd->vflag[vstage]);
                    }
                    if (two) asm volatile("bar.sync 1, 256;" ::: "memory");
                    else asm volatile("bar.sync %0, 128;" ::"r"(2 + st) : "memory");
                }
                if (active) {
                    tc_fence_after();
                    uint32_t vis[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
                    if (masked) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (tree) {
                                const int off = first + 32 * q - ctx, kk = off >> 5;
                                vis[q] = __funnelshift_r(anc_at(anc, kk), anc_at(anc, kk + 1), off & 31);
                            } else {
                                const int left = lim - (first + 32 * q);
                                vis[q] = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
                            }
                        }
                    }
                    float top[4] = {m_used, -INFINITY, -INFINITY, -INFINITY};
                    auto mask32 = [&](uint32_t *y, int q) {
                        if (masked) {
                            uint32_t v = vis[0];
                            if (q == 1) v = vis[1];
                            if (q == 2) v = vis[2];
                            if (q == 3) v = vis[3];
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!((v >> j) & 1u)) y[j] = 0xFF800000u;   // -inf
                        }
                    };
                    // Scores are read twice, 32 at a time, for the maximum and for the weights; the loops stay rolled for the sake
                    // of the instruction cache, which the block's kinds of warps share.
#pragma unroll 1
                    for (int q = 0; q < 4; q += 2) {
                        uint32_t x[32], y[32];
                        tmem_ld32(colS + q * 32, x);
                        tmem_ld32(colS + q * 32 + 32, y);
                        tc_wait_ld();
                        mask32(x, q);
                        mask32(y, q + 1);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
#pragma unroll
                            for (int u = 0; u < 4; ++u) top[u] = fmaxf(top[u], fmaxf(__uint_as_float(x[j + u]), __uint_as_float(y[j + u])));
                        }
                    }
                    const float m_new = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    // The output is rescaled only when the maximum has grown by more than 2^8: weights up to 2^8 are as
                    // exact as those up to 1, and most tiles then leave the output alone.
                    const bool grow = (m_new - m_used) * c > 8.0f;
                    if (__any_sync(0xFFFFFFFFu, grow)) {
                        const float alpha = m_new == -INFINITY ? 1.0f : ex2_fast((m_used - m_new) * c);
                        m_used = m_new;
                        l *= alpha;
                        if (k != begin) {
#pragma unroll 1
                            for (int j = 0; j < DP; j += 32) {
                                uint32_t o[32];
                                tmem_ld32(colO + j, o);
                                tc_wait_ld();
#pragma unroll
                                for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
                                tmem_st32(colO + j, o);
                            }
                        }
                    }
                    const float shift = m_used == -INFINITY ? 0.0f : m_used * c;
                    const f32x2 c2 = f2_pack(c, c), s2 = f2_pack(-shift, -shift);
                    f32x2 sum[2] = {f2_pack(l, 0.0f), f2_pack(0.0f, 0.0f)};
                    // A chunk's weights go where its scores were: upper parts, then lower ones.
                    uint32_t x[32];
                    tmem_ld32(colS, x);
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t p[32];
                        tc_wait_ld();
                        mask32(x, q);
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            const f32x2 e = f2_ex2(f2_fma(f2_from_u32x2(x[2 * u], x[2 * u + 1]), c2, s2));
                            sum[u & 1] = f2_add(sum[u & 1], e);
                            weight_parts(e, p[u], p[16 + u]);
                        }
                        if (q < 3) tmem_ld32(colS + q * 32 + 32, x);
                        tmem_st32(colS + q * 32, p);
                        if (q == 1 && !(own && masked)) {   // there the output may have to be touched before any product
                            tc_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&ms->p_half[st]);
                        }
                    }
                    l = f2_sum(f2_add(sum[0], sum[1]));
                    tc_wait_st();
                    if (own && masked) {
                        // The cleared values are added here for the rows that see them, with the weight that the product would
                        // have used.
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            uint32_t f = *reinterpret_cast<volatile uint32_t *>(&fd->vflag[vstage][q]);
                            uint32_t mine = vis[0];
                            if (q == 1) mine = vis[1];
                            if (q == 2) mine = vis[2];
                            if (q == 3) mine = vis[3];
                            while (f) {
                                const int b = __ffs(f) - 1, j = q * 32 + b;
                                f &= f - 1;
                                const uint32_t at = colS + (j & ~31) + (j & 31) / 2, pw = tmem_ld1(at), rw = tmem_ld1(at + 16);
                                tc_wait_ld();
                                const float w = j & 1 ? bf16_hi(pw) + bf16_hi(rw) : bf16_lo(pw) + bf16_lo(rw);
                                const bool sees = (mine >> b) & 1u;
                                if (first + j >= end) continue;   // flags mean nothing after a wait gave up
                                const int32_t *table = a.bt.page_table + pi->table * a.bt.table_pitch;
                                const int64_t off = slot_offset(a.c, table, first + j);
                                if (off < 0) continue;
#pragma unroll 1
                                for (int d = 0; d < a.c.head_dim; d += 32) {
                                    uint32_t o[32];
                                    tmem_ld32(colO + d, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int u = 0; u < 32; ++u) {
                                        const float vv = d + u < a.c.head_dim ? cached_value<C8>(a, off, table, first + j, pi->h, d + u) : 0.0f;
                                        if (sees) o[u] = __float_as_uint(__uint_as_float(o[u]) + w * vv);
                                    }
                                    tmem_st32(colO + d, o);
                                }
                                tc_wait_st();
                            }
                        }
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    if (!active || (own && masked)) mbar_arrive(&ms->p_half[st]);
                    mbar_arrive(&ms->p_full[st]);
                }
            }
            // ---- the piece's end
            const int nk = k1 - k0;
            const bool has1 = two || nk > 1;                     // stream 1 has scored something
            float inv, m_all = m_used, l_all = l, f0 = 1.0f, f1 = 0.0f;
            if (!two) {
                ms->ml[st][row] = make_float2(m_used, l);
                asm volatile("bar.sync 1, 256;" ::: "memory");
                const float2 o = ms->ml[st ^ 1][row];
                m_all = fmaxf(m_used, o.x);
                const float ref = m_all == -INFINITY ? 0.0f : m_all;
                const float mine = ex2_fast((m_used - ref) * c), other = ex2_fast((o.x - ref) * c);
                l_all = st == 0 ? l * mine + o.y * other : o.y * other + l * mine;
                f0 = st == 0 ? mine : other;
                f1 = st == 0 ? other : mine;
                wait_phase(fd, &ms->o_full[0], o_phases & 1);
                o_phases ^= 1;
                if (has1) {
                    wait_phase(fd, &ms->o_full[1], (o_phases >> 1) & 1);
                    o_phases ^= 2;
                }
            } else {
                wait_phase(fd, &ms->o_full[st], (o_phases >> st) & 1);
                o_phases ^= 3;   // the other stream's warps see that one
            }
            __syncwarp();
            tc_fence_after();
            if (active) {
                const int g = pi->m0 + m - i * a.G, qh = pi->h * a.G + g;
                const size_t slot = (size_t)pi->slot + m;
                const int D = a.c.head_dim;
                const bool whole = pi->whole;
                inv = l_all > 0.0f || l_all != l_all ? 1.0f / l_all : 0.0f;
                char *dst = a.out + (int64_t)(pi->r0 + i) * a.o_row + (int64_t)qh * a.o_head;
                float *part = a.part + slot * D;
                // one stream's rows: all its columns.  Both streams for the same rows: half of the columns each.
                const int d0 = two ? 0 : st * (DP / 2), d1 = two ? DP : d0 + DP / 2;
#pragma unroll 1
                for (int d = d0; d < d1; d += 32) {
                    uint32_t o[32];
                    tmem_ld32(two ? colO + d : base + kColO + d, o);
                    tc_wait_ld();
                    if (!two) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f0);
                        if (has1) {
                            uint32_t o1[32];
                            tmem_ld32(base + kColO + 128 + d, o1);
                            tc_wait_ld();
#pragma unroll
                            for (int u = 0; u < 32; ++u)
                                o[u] = __float_as_uint(fmaf(__uint_as_float(o1[u]), f1, __uint_as_float(o[u])));
                        }
                    }
                    if (m < vr) {
#pragma unroll
                        for (int u = 0; u < 32; u += 8) {
                            if (d + u >= D) continue;
                            if (whole) {
                                float f[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[u + e]) * inv;
                                *reinterpret_cast<uint4 *>(dst + (d + u) * 2) = pack16<2>(f);
                            } else {
                                *reinterpret_cast<uint4 *>(part + d + u) = make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
                                *reinterpret_cast<uint4 *>(part + d + u + 4) = make_uint4(o[u + 4], o[u + 5], o[u + 6], o[u + 7]);
                            }
                        }
                    }
                }
                if (m < vr && (two || st == 0)) {
                    if (!whole) a.part_ml[slot] = make_float2(m_all * c, l_all);
                    else if (a.lse)
                        a.lse[(size_t)(pi->r0 + i) * a.q_heads + qh] = l_all == 0.0f ? -INFINITY : (m_all * c + log2f(l_all)) / kLog2e;
                }
                tc_fence_before();
            }
            if (!two) {
                asm volatile("bar.sync 1, 256;" ::: "memory");   // both have read both outputs
                tc_fence_after();
            }
            seq += 2 * nk;
            __syncwarp();
            if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
        }
    } else if (warp < 12) {
        regs_dec<kRegsOther>();
        // ---------------------------------------------------------------- producers
        if constexpr (C8) feed8_widen<DP, S::STAGES, 128, S::SLOTS>(a, fd, f8, smem_addr(smem), smem_addr(smem) + S::OFF_KV, smem_addr(smem) + S::OFF_RAW, warp - 8, lane);
        else feed_produce<DP, S::STAGES, 128>(a, a2, fd, smem_addr(smem), smem_addr(smem) + S::OFF_KV, warp - 8, lane);
    } else {
        regs_dec<kRegsOther>();
        if (warp == 12) {   // the whole warp runs this, with uniform values
            // ------------------------------------------------------------ matrix products
            const uint32_t sbase = smem_addr(smem), tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            constexpr uint32_t shape_o = mma_shape(DP, false, true, false, false);
            uint32_t p_phases = 0, q_phases = 0, seq = 0;   // a bit a stream, a query tile
            int qnext = 0;
            for (int it = 0;; ++it) {
                const PieceInfo *pi = &fd->pd[it % kRing];
                if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1))) break;
                const int nk = __shfl_sync(0xFFFFFFFFu, pi->k1 - pi->k0, 0);
                const bool two = __shfl_sync(0xFFFFFFFFu, pi->vr, 0) > 128;
                if (nk <= 0) break;
                const int rows_from = C8 ? INT32_MAX   // the widening warps fence their tiles
                                         : __shfl_sync(0xFFFFFFFFu, a2.split ? 0 : pi->box_tiles - pi->k0, 0);   // from this tile on, copied by rows
                if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
                // Job n: stream n & 1, key tile n / 2 (two row tiles) or n.
                const int jobs = two ? 2 * nk : nk, shift = two ? 1 : 0;
                for (int t = 0; t < (two ? 2 : 1); ++t) {
                    const int qs = two ? t : qnext;
                    wait_phase(fd, &fd->q_full[qs], (q_phases >> qs) & 1);
                    q_phases ^= 1u << qs;
                }
                __syncwarp();
                fence_async_smem();
                // S = Q K^T of job n, inside elect_one; its keys have been waited for
                auto scores = [&](int n) {
                    const int s = n & 1, qs = two ? s : qnext;
                    const uint32_t stage = (seq + 2 * (n >> shift)) % S::STAGES;
                    const uint64_t q = smem_operand(sbase + qs * S::TILE, 16, 1024);
                    const uint64_t kt = smem_operand(sbase + S::OFF_KV + stage * S::TILE, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk) {
                        const uint32_t at = ((kk >> 2) * S::HALF + (kk & 3) * 32) >> 4;
                        mma_ss(tm + kColS + s * 128, q + at, kt + at, a2.shape_s, kk > 0);
                    }
                    mma_commit(&ms->s_full[s]);
                    if (!two || s == 1) mma_commit(&fd->kv_empty[stage]);
                    if (two ? n >= jobs - 2 : n == jobs - 1) mma_commit(&fd->q_empty[qs]);
                };
                auto keys_bar = [&](int n) { return &fd->kv_full[(seq + 2 * (n >> shift)) % S::STAGES]; };
                auto keys_phase = [&](int n) { return ((seq + 2 * (n >> shift)) / S::STAGES) & 1; };
                auto keys_wait = [&](int n) {
                    wait_phase(fd, keys_bar(n), keys_phase(n));
                    __syncwarp();
                    if ((n >> shift) >= rows_from) fence_async_smem();
                    tc_fence_after();
                };
                for (int n = 0; n < min(jobs, 2); ++n) {
                    keys_wait(n);
                    if (elect_one()) scores(n);
                    __syncwarp();
                }
                for (int n = 0; n < jobs; ++n) {   // O += P V of job n, and S of the stream's next job right behind it
                    const int s = n & 1, tile = n >> shift;
                    const uint32_t vs = seq + 2 * tile + 1, stage = vs % S::STAGES;
                    const uint64_t v = smem_operand(sbase + S::OFF_KV + stage * S::TILE, S::HALF, 1024);
                    const uint32_t o = tm + kColO + s * 128, w = tm + kColS + s * 128, phase = (p_phases >> s) & 1;
                    p_phases ^= 1u << s;
                    // The next keys are looked at before the weights are waited for: where they are there, nothing stands between
                    // the two groups of products.
                    const bool next = n + 2 < jobs;
                    bool ready = next && __all_sync(0xFFFFFFFFu, mbar_test_wait(keys_bar(n + 2), keys_phase(n + 2)));
                    if (ready && ((n + 2) >> shift) >= rows_from) fence_async_smem();
                    wait_phase(fd, &fd->kv_full[stage], (vs / S::STAGES) & 1);
                    // Half of the tokens at a time, so that one half's products run while the other's weights are made; of each
                    // the weights' upper parts, then the lower ones.
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        wait_phase(fd, half ? &ms->p_full[s] : &ms->p_half[s], phase);
                        __syncwarp();
                        if (half == 0 && tile >= rows_from) fence_async_smem();
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int part = 0; part < 2; ++part)
#pragma unroll
                                for (int kk = half * 4; kk < half * 4 + 4; ++kk)
                                    mma_ts(o, w + (kk >> 1) * 32 + part * 16 + (kk & 1) * 8, v + kk * (2048 >> 4), shape_o, 1u);
                            if (half) {
                                if (!two || s == 1) mma_commit(&fd->kv_empty[stage]);
                                if (n + 2 >= jobs) mma_commit(&ms->o_full[s]);
                                if (ready) scores(n + 2);
                            }
                        }
                        __syncwarp();
                    }
                    if (next && !ready) {
                        keys_wait(n + 2);
                        if (elect_one()) scores(n + 2);
                        __syncwarp();
                    }
                }
                if (!two) qnext ^= 1;
                seq += 2 * nk;
            }
            if (elect_one()) mma_commit(&ms->done);
            wait_phase<true>(fd, &ms->done, 0);   // the products end by themselves
            __syncwarp();
        } else if (warp == 13) {
            // ------------------------------------------------------------ the walk
            feed_walk(a, a2, fd, ms->walk, lane);
        } else if constexpr (C8) {
            feed8_load<DP, kRawTokens, S::SLOTS, true, false, false>(a, a2, fd, f8, smem_addr(smem) + S::OFF_RAW + (warp - 14) * (S::SLOTS * kRawTokens * DP), warp - 14, lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && fd->dead) {
        if constexpr (C8) feed8_drain<S::SLOTS>(fd, f8, a.stats);
        else feed_drain<S::STAGES>(fd, a.stats);
    }
    if (warp == 12) tmem_free(tmem, 512);
}

template <int DP, bool C8>
cudaError_t run_tall(AttendArgs &a, bool negate, cudaStream_t stream) {
    constexpr size_t bytes = TallShape<DP, C8>::OFF_MISC + (C8 ? sizeof(TallShared8) : sizeof(TallShared));
    static_assert(bytes <= 232448, "shared memory of a block");
    if (prepare_kernel((const void *)k_attend_tall<DP, C8>, kTcThreads, bytes) < 1) return cudaErrorInvalidConfiguration;
    const uint32_t shape = mma_shape(128, false, false, negate, false);
    static_assert(kTilesTall.TM == kTallRows && kTilesTall.TK == kTcKeys, "the cutting's tiles are the kernel's");
    a.geo.set(kTilesTall);
    k_attend_tall<DP, C8><<<a.geo.blocks, kTcThreads, bytes, stream>>>(a, C8 ? tc_args8(a.c, DP, false, shape) : tc_args(a.c, shape));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_tall(AttendArgs &a, cudaStream_t stream) {
    AttendArgs t = a;
    // The maximum is taken of q.k before the scale, so the scale has to be positive: a negative one negates the queries in the
    // product, and zero becomes the smallest normal number, which tells weights apart only where q.k passes 10^36.
    const bool negate = a.scale_log2 < 0.0f;
    t.scale_log2 = fmaxf(fabsf(a.scale_log2), FLT_MIN);
    const bool narrow = a.c.head_dim <= 64;
    const cudaError_t e = a.sc.k ? (narrow ? run_tall<64, true>(t, negate, stream) : run_tall<128, true>(t, negate, stream))
                                 : (narrow ? run_tall<64, false>(t, negate, stream) : run_tall<128, false>(t, negate, stream));
    a.geo = t.geo;
    return e;
}

}  // namespace sv
