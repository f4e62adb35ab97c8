// sv_attend_tc.cu — sv_kv_attend on the tensor cores: bf16, heads up to 128 wide.
//
// A persistent block of 16 warps walks its range of (unit, key tile)s; units are 256 packed rows, key tiles 128 tokens.
//   warps 0-3, 4-7   softmax of two streams: a thread owns one row of 128 scores in tensor memory
//   warps 8-11       producers: gather keys, values and queries from their pages into swizzled shared memory
//   warp 12          one thread issues the matrix products
//   warp 13          walks the range and describes the pieces to the others, a few ahead
// Streams.  A piece of more than 128 rows is two row tiles that share each key tile, one a stream.  A piece of up to 128 rows
// is one row tile whose even key tiles go to one stream and odd ones to the other, each with its own maximum, sum and
// output, added at the piece's end.  Either way one stream's products run while the other's softmax does.
// Tensor memory (512 columns): scores 2 x 128, the weights over the scores they came from, outputs 2 x 128.
// Weights.  A weight enters the product with V as two bf16 parts, its rounding and what that left (16 bits in all): one
// part alone is off by 2^-8, as much as the rounding of the output.
#include "sv_attend.cuh"
#include "sv_tc.cuh"

namespace sv {

namespace {

constexpr int kTcThreads = 512;
constexpr int kTcRows = 256, kTcKeys = 128;
constexpr int kRing = 3;              // piece descriptions in flight
constexpr int kTcWait = 13;           // warps that read a piece description
constexpr int kNoPage = INT32_MIN;     // a token past the unit's last
constexpr uint32_t kColS = 0, kColO = 256;

struct PieceInfo {
    long long slot;                   // first workspace slot
    int r0, m0, vr, h;                // segment's first row, first packed row, rows, key head
    int table, key0, ctx, end;        // page table's sequence, tokens
    int k0, k1;                       // key tiles; k0 == k1: no more pieces
    int own, tree, whole, boxes;      // own segment, tree mask, output complete here, full tiles load as boxes
    uint8_t par[SV_MAX_TREE];         // a tree's parents (255: invalid)
};

template <int DP>
struct TcShape {
    static constexpr int TILE = 128 * DP * 2;              // bytes of 128 rows
    static constexpr int STAGES = DP == 128 ? 5 : 8;
    static constexpr int HALF = 128 * 128;                 // bytes of 128 rows of 64 elements
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_MISC = OFF_KV + STAGES * TILE;
};

struct Misc {
    uint64_t kv_full[8], kv_empty[8], q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], pd_full[kRing], pd_empty[kRing], done;
    PieceInfo pd[kRing];
    uint32_t vflag[8][4];             // per stage: tokens whose values are not finite (last tiles of a sequence only)
    union {
        struct {
            Walk walk;                // read before the first piece is described
            long long warp_sum[kTcThreads / 32];
        };
        float2 ml[2][128];            // maxima and sums exchanged by the streams
    };
    uint32_t tmem;
    int dead;                         // a wait gave up: nobody waits any more
};

// Waits for a phase.  Gives up for everybody after the library's limit: waits return at once from then on, the block
// runs to its end with meaningless results and the error is reported.
__device__ __forceinline__ void wait_phase(Misc *ms, uint64_t *bar, uint32_t parity, sv_stats *stats) {
    if (mbar_try_wait(bar, parity)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait_sleep(bar, parity, kSuspendHintNs)) {
        if (*reinterpret_cast<volatile int *>(&ms->dead)) return;
        if (clock64() - t0 > kWaitLimitCycles) {
            *reinterpret_cast<volatile int *>(&ms->dead) = 1;
            report_error(stats, SV_ERR_TIMEOUT, -1);
            return;
        }
    }
}

__device__ __forceinline__ bool not_finite16(uint4 w) {
    auto bad = [](uint32_t x) { return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u; };
    return bad(w.x) || bad(w.y) || bad(w.z) || bad(w.w);
}

// Asynchronous copies in flight, oldest first, each with the barrier it completes (one arrival a warp).
struct CopyQueue {
    uint64_t bars = 0;   // barrier numbers, 8 bits each
    int n = 0;

    __device__ __forceinline__ void retire(uint64_t *base, int lane) {
        switch (n - 1) {
            case 0: cp_async_wait<0>(); break;
            case 1: cp_async_wait<1>(); break;
            case 2: cp_async_wait<2>(); break;
            case 3: cp_async_wait<3>(); break;
            case 4: cp_async_wait<4>(); break;
            case 5: cp_async_wait<5>(); break;
            case 6: cp_async_wait<6>(); break;
            default: cp_async_wait<7>(); break;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + (bars & 0xFF));
        bars >>= 8;
        --n;
    }
    __device__ __forceinline__ void add(uint64_t *base, int bar, int lane) {
        cp_async_commit();
        if (n == 8) retire_full(base, lane);
        bars |= (uint64_t)bar << (8 * n);
        ++n;
    }
    __device__ __forceinline__ void retire_full(uint64_t *base, int lane) {
        cp_async_wait<8>();   // the group just committed is the ninth
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + (bars & 0xFF));
        bars >>= 8;
        --n;
    }
};

__device__ __forceinline__ uint32_t bf16_pair(f32x2 x) {
    float lo, hi;
    uint32_t w;
    f2_unpack(x, lo, hi);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// Bits of the 128 tokens first .. first + 127 that a row of a tree sees, from its ancestor bits.
__device__ __forceinline__ uint32_t anc_at(const uint32_t (&anc)[5], int k) {
    if (k < 0) return 0xFFFFFFFFu;   // cached tokens
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i)
        if (i == k) w = anc[i];
    return w;
}

// Keys and values as 4-D tensors (element, head, slot, page) with boxes of 64 elements by box_rows slots, loaded with the
// 128-byte swizzle; box_rows is 0 where a box could not stay inside a page.
struct TcArgs {
    CUtensorMap k, v;
    int box_rows;
    uint32_t shape_s;     // of the score product
};

template <int DP>
__global__ void __launch_bounds__(kTcThreads, 1) k_attend_tc(const __grid_constant__ AttendArgs a, const __grid_constant__ TcArgs a2) {
    using S = TcShape<DP>;
    extern __shared__ __align__(1024) char smem[];
    Misc *ms = reinterpret_cast<Misc *>(smem + S::OFF_MISC);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

    if (smem_addr(smem) & 1023) {   // the swizzle goes by address bits
        if (tid == 0) report_error(a.stats, SV_ERR_CUDA, -1);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&ms->kv_full[i], 4);
            mbar_init(&ms->kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms->q_full[i], 4);
            mbar_init(&ms->q_empty[i], 1);
            mbar_init(&ms->s_full[i], 1);
            mbar_init(&ms->p_full[i], 4);
            mbar_init(&ms->o_full[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&ms->pd_full[i], 1);
            mbar_init(&ms->pd_empty[i], kTcWait);
        }
        mbar_init(&ms->done, 1);
        ms->dead = 0;
        fence_barrier_init();
    }
    if (warp == 12) tmem_alloc(&ms->tmem, 512);
    tc_fence_before();
    walk_start<kTcThreads>(a, &ms->walk, ms->warp_sum);   // has block-wide barriers
    tc_fence_after();
    const uint32_t tmem = ms->tmem;

    if (warp < 8) {
        regs_inc<176>();
        // ---------------------------------------------------------------- softmax
        const int st = warp >> 2;                               // stream
        const int wl = warp & 3, row = wl * 32 + lane;          // tensor-memory lane
        const uint32_t base = tmem + ((uint32_t)(wl * 32) << 16);
        const uint32_t colS = base + kColS + st * 128, colO = base + kColO + st * 128;
        uint32_t s_phase = 0, o_phase[2] = {0, 0}, seq = 0;
        const float c = a.scale_log2;
        for (int it = 0;; ++it) {
            PieceInfo *pi = &ms->pd[it % kRing];
            wait_phase(ms, &ms->pd_full[it % kRing], (it / kRing) & 1, a.stats);
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
                wait_phase(ms, &ms->s_full[st], s_phase, a.stats);
                s_phase ^= 1;
                __syncwarp();
                if (active) {
                    tc_fence_after();
                    uint32_t x[128];
#pragma unroll
                    for (int j = 0; j < 128; j += 32) tmem_ld32(colS + j, x + j);
                    const int first = key0 + k * kTcKeys;
                    const bool masked = own ? first + kTcKeys > ctx : first + kTcKeys > end;
                    tc_wait_ld();
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
#pragma unroll
                        for (int j = 0; j < 128; ++j)
                            if (!((vis[j >> 5] >> (j & 31)) & 1u)) x[j] = 0xFF800000u;   // -inf
                    }
                    float top[4] = {m_used, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < 128; j += 8) {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            top[u] = fmaxf(top[u], fmaxf(__uint_as_float(x[j + 2 * u]), __uint_as_float(x[j + 2 * u + 1])));
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
                    const f32x2 minus1 = f2_pack(-1.0f, -1.0f);
                    f32x2 sum[2] = {f2_pack(l, 0.0f), f2_pack(0.0f, 0.0f)};
#pragma unroll
                    for (int j = 0; j < 128; j += 64) {
                        uint32_t p[32], r[32];
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            const f32x2 e = f2_ex2(f2_fma(f2_from_u32x2(x[j + 2 * u], x[j + 2 * u + 1]), c2, s2));
                            sum[u & 1] = f2_add(sum[u & 1], e);
                            p[u] = bf16_pair(e);
                            r[u] = bf16_pair(f2_fma(f2_from_bf16x2(p[u]), minus1, e));
                        }
                        tmem_st32(colS + j / 2, p);
                        tmem_st32(colS + 64 + j / 2, r);
                    }
                    l = f2_sum(f2_add(sum[0], sum[1]));
                    tc_wait_st();
                    if (own && masked) {
                        // Values that are not finite were replaced by zeros on the way in; they are added here for the rows
                        // that see them, with the weight that the product would have used.
                        const uint32_t vs = seq + 2 * (k - k0) + 1, stage = vs % S::STAGES;
                        wait_phase(ms, &ms->kv_full[stage], (vs / S::STAGES) & 1, a.stats);
                        __syncwarp();
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            uint32_t f = *reinterpret_cast<volatile uint32_t *>(&ms->vflag[stage][q]);
                            uint32_t mine = vis[0];
                            if (q == 1) mine = vis[1];
                            if (q == 2) mine = vis[2];
                            if (q == 3) mine = vis[3];
                            while (f) {
                                const int b = __ffs(f) - 1, j = q * 32 + b;
                                f &= f - 1;
                                const uint32_t pw = tmem_ld1(colS + j / 2), rw = tmem_ld1(colS + 64 + j / 2);
                                tc_wait_ld();
                                const float w = j & 1 ? bf16_hi(pw) + bf16_hi(rw) : bf16_lo(pw) + bf16_lo(rw);
                                const bool sees = (mine >> b) & 1u;
                                const int64_t off = slot_offset(a.c, a.bt.page_table + pi->table * a.bt.table_pitch, first + j);
                                const char *v = a.c.v + off + pi->h * a.c.head_b;
#pragma unroll 1
                                for (int d = 0; d < a.c.head_dim; d += 32) {
                                    uint32_t o[32];
                                    tmem_ld32(colO + d, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int u = 0; u < 32; ++u) {
                                        const float vv = d + u < a.c.head_dim
                                                             ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(v)[d + u] << 16)
                                                             : 0.0f;
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
                if (lane == 0) mbar_arrive(&ms->p_full[st]);
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
                wait_phase(ms, &ms->o_full[0], o_phase[0], a.stats);
                o_phase[0] ^= 1;
                if (has1) {
                    wait_phase(ms, &ms->o_full[1], o_phase[1], a.stats);
                    o_phase[1] ^= 1;
                }
            } else {
                wait_phase(ms, &ms->o_full[st], o_phase[st], a.stats);
                o_phase[st] ^= 1;
                o_phase[st ^ 1] ^= 1;   // the other stream's warps see that one
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
            if (lane == 0) mbar_arrive(&ms->pd_empty[it % kRing]);
        }
    } else if (warp < 12) {
        regs_dec<80>();
        // ---------------------------------------------------------------- producers
        const int wl = warp - 8;
        uint64_t *bars = ms->kv_full;
        const int bar_q = (int)(ms->q_full - ms->kv_full);
        const uint32_t sbase = smem_addr(smem);
        const int D = a.c.head_dim;
        constexpr int CH = DP / 8;            // 16-byte chunks of a row
        constexpr int RP = 32 / CH;           // rows of a warp's pass
        const int ch = lane % CH, rsub = lane / CH;
        const bool real = ch * 8 < D;         // chunks past the head are zero
        CopyQueue cq;
        uint32_t seq = 0, q_use[2] = {0, 0};
        int qnext = 0;
        // Waits for a barrier and passes on the copies that land meanwhile: whoever completes the barrier may be waiting for them.
        auto acquire = [&](uint64_t *bar, uint32_t parity) {
            // A test, not a try: a try may suspend the warp for microseconds, and copies that land meanwhile have to be
            // passed on.  The whole warp takes one way: lanes may see the phase end at different tests.
            while (!__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity))) {
                if (cq.n == 0) {
                    wait_phase(ms, bar, parity, a.stats);
                    return;
                }
                cq.retire(bars, lane);
            }
        };
        // destination of this lane's chunk of row r (r & 7 is the swizzle)
        auto place = [&](uint32_t tile, int r) { return tile + (ch >> 3) * S::HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4); };
        for (int it = 0;; ++it) {
            const PieceInfo *pi = &ms->pd[it % kRing];
            acquire(&ms->pd_full[it % kRing], (it / kRing) & 1);
            const int k0 = pi->k0, k1 = pi->k1;
            if (k0 >= k1) break;
            const int vr = pi->vr, key0 = pi->key0, end = pi->end, ctx = pi->ctx, own = pi->own, h = pi->h, m0 = pi->m0, r0 = pi->r0, pi_boxes = pi->boxes;
            const int32_t *table = a.bt.page_table + pi->table * a.bt.table_pitch;
            const int tab = pi->table;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms->pd_empty[it % kRing]);
            const bool two = vr > 128;
            // A tile that every row sees whole goes as boxes where it can, the others by rows: a lane's token of a tile, and its
            // page, are those of the lane's box or row.
            const int boxes = pi_boxes ? 32 / a2.box_rows : 0;
            auto by_box = [&](int k) { return boxes > 0 && key0 + (k + 1) * kTcKeys <= (own ? ctx : end); };
            auto key_of = [&](int k) { return key0 + k * kTcKeys + wl * 32 + (by_box(k) ? lane * a2.box_rows : lane); };
            auto page_of = [&](int k) {
                if (by_box(k) && lane >= boxes) return kNoPage;
                const int key = key_of(k);
                return key < end ? table[key / a.c.page_size] : kNoPage;
            };
            int page = page_of(k0);
            // queries
            for (int t = 0; t < (two ? 2 : 1); ++t) {
                const int qs = two ? t : qnext;
                acquire(&ms->q_empty[qs], (q_use[qs] & 1) ^ 1);
                ++q_use[qs];
                const int m = t * 128 + wl * 32 + lane;
                int64_t off = -1;
                if (m < vr) {
                    const int r = (m0 + m) / a.G;
                    off = (int64_t)(r0 + r) * a.q_row + (int64_t)(h * a.G + (m0 + m - r * a.G)) * a.q_head;
                }
                const uint32_t tile = sbase + qs * S::TILE;
#pragma unroll
                for (int p = 0; p < 32 / RP; ++p) {
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, p * RP + rsub);
                    const bool ok = o >= 0 && real;
                    cp_async16(place(tile, wl * 32 + p * RP + rsub), a.q + (ok ? o + ch * 16 : 0), ok);
                }
                cq.add(bars, bar_q + qs, lane);
            }
            if (!two) qnext ^= 1;
            for (int k = k0; k < k1; ++k) {
                const int key = key_of(k), pg = page, slot = key - key / a.c.page_size * a.c.page_size;
                const bool box = by_box(k);
                int64_t off = -1;
                if (pg >= 0 && pg < a.c.n_pages) off = pg * a.c.page_b + slot * a.c.slot_b + h * a.c.head_b;
                else if (pg != kNoPage) report_error(a.stats, SV_ERR_INVALID_ARG, tab);
                if (k + 1 < k1) page = page_of(k + 1);
                const bool masked = own && key0 + (k + 1) * kTcKeys > ctx;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t stage = seq % S::STAGES;
                    acquire(&ms->kv_empty[stage], ((seq / S::STAGES) & 1) ^ 1);
                    ++seq;
                    const uint32_t tile = sbase + S::OFF_KV + stage * S::TILE;
                    const char *src = kv ? a.c.v : a.c.k;
                    if (box) {   // a bad page id lies outside the tensor and reads zeros
                        if (elect_one()) mbar_arrive_expect_tx(&ms->kv_full[stage], 32 * DP * 2);
                        __syncwarp();
                        for (int b = 0; b < boxes; ++b) {
                            const int bp = __shfl_sync(0xFFFFFFFFu, pg, b), bs = __shfl_sync(0xFFFFFFFFu, slot, b);
                            const uint32_t dst = tile + (wl * 32 + b * a2.box_rows) * 128;
                            if (elect_one()) {
                                const CUtensorMap *map = kv ? &a2.v : &a2.k;
                                box_load(dst, map, &ms->kv_full[stage], 0, h, bs, bp);
                                if (DP == 128) box_load(dst + S::HALF, map, &ms->kv_full[stage], 64, h, bs, bp);
                            }
                            __syncwarp();
                        }
                        continue;
                    }
                    if (kv == 1 && masked) {
                        // values through registers: a token whose values are not all finite goes in as zeros and is flagged
                        uint32_t flags = 0;
#pragma unroll
                        for (int p4 = 0; p4 < 32 / RP; p4 += 4) {
                            uint4 w[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int64_t o = __shfl_sync(0xFFFFFFFFu, off, (p4 + u) * RP + rsub);
                                w[u] = make_uint4(0, 0, 0, 0);
                                if (o >= 0 && real) w[u] = *reinterpret_cast<const uint4 *>(src + o + ch * 16);
                            }
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const uint32_t bad = __ballot_sync(0xFFFFFFFFu, not_finite16(w[u]));
#pragma unroll
                                for (int g = 0; g < RP; ++g) {
                                    const bool b = (bad >> (g * CH)) & (CH == 32 ? 0xFFFFFFFFu : (1u << CH) - 1u);
                                    if (b) flags |= 1u << ((p4 + u) * RP + g);
                                    if (b && rsub == g) w[u] = make_uint4(0, 0, 0, 0);
                                }
                                const uint32_t dst = place(tile, wl * 32 + (p4 + u) * RP + rsub);
                                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(w[u].x), "r"(w[u].y), "r"(w[u].z),
                                             "r"(w[u].w)
                                             : "memory");
                            }
                        }
                        if (lane == 0) ms->vflag[stage][wl] = flags;
                    } else {
#pragma unroll
                        for (int p = 0; p < 32 / RP; ++p) {
                            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, p * RP + rsub);
                            const bool ok = o >= 0 && real;
                            cp_async16(place(tile, wl * 32 + p * RP + rsub), src + (ok ? o + ch * 16 : 0), ok);
                        }
                    }
                    cq.add(bars, (int)stage, lane);
                }
            }
        }
        while (cq.n) cq.retire(bars, lane);
    } else {
        regs_dec<80>();
        if (warp == 12) {   // the whole warp runs this, with uniform values
            // ------------------------------------------------------------ matrix products
            const uint32_t sbase = smem_addr(smem), tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            constexpr uint32_t shape_o = mma_shape(DP, true, false);
            uint32_t p_phase[2] = {0, 0}, seq = 0, q_use[2] = {0, 0};
            int qnext = 0;
            for (int it = 0;; ++it) {
                const PieceInfo *pi = &ms->pd[it % kRing];
                wait_phase(ms, &ms->pd_full[it % kRing], (it / kRing) & 1, a.stats);
                __syncwarp();
                const int nk = __shfl_sync(0xFFFFFFFFu, pi->k1 - pi->k0, 0);
                const bool two = __shfl_sync(0xFFFFFFFFu, pi->vr, 0) > 128;
                if (nk <= 0) break;
                if (lane == 0) mbar_arrive(&ms->pd_empty[it % kRing]);
                const int jobs = two ? 2 * nk : nk;
                auto weigh = [&](int n) {   // O += P V of job n
                    const int s = n & 1, tile = two ? n >> 1 : n;
                    const uint32_t vs = seq + 2 * tile + 1, stage = vs % S::STAGES;
                    wait_phase(ms, &ms->kv_full[stage], (vs / S::STAGES) & 1, a.stats);
                    wait_phase(ms, &ms->p_full[s], p_phase[s], a.stats);
                    p_phase[s] ^= 1;
                    __syncwarp();
                    tc_fence_after();
                    const uint64_t v = smem_operand(sbase + S::OFF_KV + stage * S::TILE, S::HALF, 1024);
                    const uint32_t o = tm + kColO + s * 128, w = tm + kColS + s * 128;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 16; ++kk)   // the weights' upper parts, then the lower ones
                            mma_ts(o, w + kk * 8, v + (kk & 7) * (2048 >> 4), shape_o, 1u);
                        if (!two || s == 1) mma_commit(&ms->kv_empty[stage]);
                        if (n + 2 >= jobs) mma_commit(&ms->o_full[s]);
                    }
                    __syncwarp();
                };
                for (int n = 0; n < jobs; ++n) {
                    const int s = n & 1, tile = two ? n >> 1 : n;
                    const int qs = two ? s : qnext;
                    const uint32_t ks = seq + 2 * tile, stage = ks % S::STAGES;
                    if (n == 0 || (two && n == 1)) {
                        wait_phase(ms, &ms->q_full[qs], q_use[qs] & 1, a.stats);
                        ++q_use[qs];
                    }
                    wait_phase(ms, &ms->kv_full[stage], (ks / S::STAGES) & 1, a.stats);
                    __syncwarp();
                    tc_fence_after();
                    const uint64_t q = smem_operand(sbase + qs * S::TILE, 16, 1024);
                    const uint64_t kt = smem_operand(sbase + S::OFF_KV + stage * S::TILE, 16, 1024);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < DP / 16; ++kk) {
                            const uint32_t at = ((kk >> 2) * S::HALF + (kk & 3) * 32) >> 4;
                            mma_ss(tm + kColS + s * 128, q + at, kt + at, a2.shape_s, kk > 0);
                        }
                        mma_commit(&ms->s_full[s]);
                        if (!two || s == 1) mma_commit(&ms->kv_empty[stage]);
                        if (two ? n >= jobs - 2 : n == jobs - 1) mma_commit(&ms->q_empty[qs]);
                    }
                    __syncwarp();
                    if (n > 0) weigh(n - 1);
                }
                weigh(jobs - 1);
                if (!two) qnext ^= 1;
                seq += 2 * nk;
            }
            if (elect_one()) mma_commit(&ms->done);
            wait_phase(ms, &ms->done, 0, a.stats);
            __syncwarp();
        } else if (warp == 13) {
            // ------------------------------------------------------------ the walk
            Walk w = ms->walk;
            for (int it = 0;; ++it) {
                Piece p;
                const bool more = w.next(a, p);
                wait_phase(ms, &ms->pd_empty[it % kRing], ((it / kRing) & 1) ^ 1, a.stats);
                PieceInfo *pi = &ms->pd[it % kRing];
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
                        pi->slot = (long long)(unit_slot(a, p.g, !own, p.h, p.t) + (size_t)blockIdx.x * kTcRows);
                        pi->r0 = p.g.r0;
                        pi->m0 = p.t * kTcRows;
                        pi->vr = p.vr;
                        pi->h = p.h;
                        pi->table = p.g.table;
                        pi->key0 = p.g.key0;
                        pi->ctx = p.g.ctx;
                        pi->end = p.end;
                        pi->boxes = a2.box_rows > 0 && p.g.key0 % a2.box_rows == 0;
                        pi->k0 = p.k0;
                        pi->k1 = p.k1;
                        pi->own = own;
                        pi->tree = tree;
                        pi->whole = p.k0 == 0 && p.k1 == p.kt && own && seg_alone(p.g);
                    } else {
                        pi->k0 = pi->k1 = 0;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms->pd_full[it % kRing]);
                if (!more) break;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_free(tmem, 512);
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
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

bool cache_map(CUtensorMap *map, char *base, const KvCache &c, int box_rows) {
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.kv_heads, (cuuint64_t)c.page_size, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.head_b, (cuuint64_t)c.slot_b, (cuuint64_t)c.page_b};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1}, one[4] = {1, 1, 1, 1};
    return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP>
sv_status run_tc(AttendArgs &a, const DeviceInfo &di, bool negate, cudaStream_t stream) {
    constexpr size_t bytes = TcShape<DP>::OFF_MISC + sizeof(Misc);
    static_assert(bytes <= 232448, "shared memory of a block");
    if (prepare_kernel((const void *)k_attend_tc<DP>, kTcThreads, bytes) < 1) return SV_ERR_CUDA;
    a.TM = kTcRows;
    a.TK = kTcKeys;
    a.blocks = di.sms;
    TcArgs a2{};
    a2.shape_s = mma_shape(128, false, negate);
    // Boxes of up to 32 slots (a producer warp's share of a tile), whole swizzle groups of 8 rows, that never cross a page.
    const int ps = a.c.page_size;
    if (ps >= 32 ? ps % 32 == 0 : ps == 8 || ps == 16) {
        a2.box_rows = ps < 32 ? ps : 32;
        if (encode_tiled() == nullptr || !cache_map(&a2.k, a.c.k, a.c, a2.box_rows) || !cache_map(&a2.v, a.c.v, a.c, a2.box_rows))
            a2.box_rows = 0;
    }
    k_attend_tc<DP><<<a.blocks, kTcThreads, bytes, stream>>>(a, a2);
    if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
    return cuda_status(launch_attend_join(a, 2, stream));
}

}  // namespace

sv_status launch_attend_tc(AttendArgs a, const DeviceInfo &di, cudaStream_t stream) {
    // The maximum is taken of q.k before the scale, so the scale has to be positive: a negative one negates the queries in the
    // product, and zero becomes a number too small to tell weights apart.
    const bool negate = a.scale_log2 < 0.0f;
    a.scale_log2 = fmaxf(fabsf(a.scale_log2), 1e-30f);
    return a.c.head_dim <= 64 ? run_tc<64>(a, di, negate, stream) : run_tc<128>(a, di, negate, stream);
}

}  // namespace sv
