// sv_attend_few.cu — sv_kv_attend on the tensor cores for up to 32 packed rows a sequence and key head (a single token or a drafted
// block times the query heads that share a key head): bf16, heads up to 128 wide.
//
// Few rows leave a tile of 128 rows mostly empty, so the products are turned round: tokens lie along the 128 rows of tensor
// memory and the packed rows along its columns,
//   S^T [128 tokens][32] = K Q^T          O^T [head element][32 + 32] += V^T [P high | P low]
// with V as stored (its contiguous axis is not the one summed over) and P^T written by the softmax to shared memory, one token's
// 32 weights a row.  A thread owns a token and its 32 scores: 32 exponentials a tile instead of 128, none of them for empty
// rows.  A weight enters as two bf16 parts (16 bits in all; one part alone is off by 2^-8, as much as the rounding of the output):
// they are two halves of the product's columns and cost no further read of V, which bounds it.
//
// The maximum of a row is kept until a score passes it by 2^8: then, and on a piece's first tile, the four warps exchange theirs and
// the output is rescaled.  Other tiles need one vote.
//
// A persistent block of 16 warps.  Warps 0-3 take a piece's even tiles and warps 4-7 its odd ones, each group with its own maxima,
// sums and output, which are added at the piece's end; 8-11 produce, 12 issues the products, 13 walks the range.
// Tensor memory (256 columns): scores 2 groups x 2 tiles x 32, outputs 2 groups x 64.
//
// What bounds it: memory.  A tile is 64 KB (heads of 128), 2800 cycles of an SM's share of the measured copy bandwidth; its
// products take about 700 and its softmax about 1300, which the two groups share.  512 sequences x 6 rows, 8 key heads, 1,024 to
// 2,048 tokens: 525 us, 6.3 TB/s or 0.92 of the measured copy bandwidth (the tall kernel: 1,040 us).
#include "sv_attend_feed.cuh"

namespace sv {

namespace {

constexpr int NR = kFewRows;
constexpr int kFewReaders = 13;       // warps that read a piece description
constexpr float kNoMax = -1e30f;      // maximum of a row that has seen no token yet

template <int DP>
struct FewShape {
    static constexpr int TILE = 128 * DP * 2;
    static constexpr int STAGES = DP == 128 ? 5 : 8;
    static constexpr int HALF = 128 * 128;
    static constexpr int OFF_P = 2 * NR * DP * 2;                 // after two query tiles
    static constexpr int PBUF = 128 * 4 * NR;                     // a group's weights: 128 tokens x (32 high + 32 low)
    static constexpr int OFF_KV = OFF_P + 2 * PBUF;
    static constexpr int OFF_MISC = OFF_KV + STAGES * TILE;
};

struct FewShared {
    Feed fd;
    uint64_t s_full[2][2], p_full[2], p_done[2], done;
    Walk walk;
    long long warp_sum[kTcThreads / 32];
    // per group
    float top[2][4][NR];              // the warps' maxima of a row, later their sums
    alignas(16) float shift[2][NR];   // minus a row's maximum (of scale * log2(e) * q.k)
    alignas(16) float zero[NR];
    int64_t to[2][NR];                // where a row's output goes (the first's, where both groups work on the piece)
    alignas(16) float alpha[2][NR];   // what a new maximum scales the row by; at the end what the group's output is scaled by
};

// Element-wise reduction of x[0..31] over the warp's lanes: lane r gets that of x[r].
template <class F>
__device__ __forceinline__ float reduce_rows(float (&x)[NR], int lane, F f) {
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < w) {
                const float mine = up ? x[i + w] : x[i], other = up ? x[i] : x[i + w];
                x[i] = f(mine, __shfl_xor_sync(0xFFFFFFFFu, other, w));
            }
        }
    }
    return x[0];
}

// The packed rows of a unit that see token `key`, as bits.
__device__ __forceinline__ uint32_t rows_that_see(const PieceInfo *pi, int key, int G, int n) {
    if (key >= pi->end) return 0;
    const int rel = key - pi->ctx;
    if (rel <= 0) return 0xFFFFFFFFu;
    if (!pi->tree) return rel * G >= 32 ? 0u : 0xFFFFFFFFu << (rel * G);
    uint32_t below = 1u << rel, rows = 0;   // the node and what descends from it: parents come before their children
    for (int i = rel + 1; i < n; ++i) {
        const int p = pi->par[i - 1];
        if (p != 255 && ((below >> p) & 1u)) below |= 1u << i;
    }
    const uint32_t heads = G >= 32 ? 0xFFFFFFFFu : (1u << G) - 1u;
    for (int i = rel; i < n; ++i)
        if ((below >> i) & 1u) rows |= heads << (i * G);
    return rows;
}

template <int DP>
__global__ void __launch_bounds__(kTcThreads, 1) k_attend_few(const __grid_constant__ AttendArgs a, const __grid_constant__ TcArgs a2) {
    using S = FewShape<DP>;
    extern __shared__ __align__(1024) char smem[];
    FewShared *ms = reinterpret_cast<FewShared *>(smem + S::OFF_MISC);
    Feed *fd = &ms->fd;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

    if (smem_addr(smem) & 1023) {   // the swizzle goes by address bits
        if (tid == 0) report_error(a.stats, SV_ERR_CUDA, -1);
        return;
    }
    if (tid == 0) {
        feed_init(fd, a, kFewReaders);
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
    if (warp == 12) tmem_alloc(&fd->tmem, 256);
    tc_fence_before();
    walk_start<kTcThreads>(a, &ms->walk, ms->warp_sum);   // has block-wide barriers
    pdl_trigger();
    tc_fence_after();
    const uint32_t tmem = fd->tmem;
    const uint32_t sbase = smem_addr(smem);

    if (warp < 8) {
        regs_inc<kRegsSoftmax>();
        // ---------------------------------------------------------------- softmax
        const int gr = warp >> 2, wl = warp & 3, t = wl * 32 + lane;   // group, warp of it, token of the tile (head element at the end)
        const uint32_t base = tmem + ((uint32_t)(wl * 32) << 16);
        const uint32_t colO = base + 128 + gr * 64;
        const uint32_t prow = sbase + S::OFF_P + gr * S::PBUF + t * (4 * NR);     // this token's weights
        const f32x2 c2 = f2_pack(a.scale_log2, a.scale_log2);
        uint32_t u = 0;   // tiles this group has worked on
        int rests = 0;    // the group that left the last piece of one tile to the other
        auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + gr) : "memory"); };
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
                    if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
                    continue;
                }
            }
            const int key0 = pi->key0, ctx = pi->ctx;
            {
                uint32_t zero[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) zero[j] = 0;
                tmem_st32(colO, zero);
                tmem_st32(colO + 32, zero);
                tc_wait_st();
            }
            f32x2 l[NR / 2];   // this token column's sums
#pragma unroll
            for (int r = 0; r < NR / 2; ++r) l[r] = 0;
            float *shift = ms->shift[gr], *alpha = ms->alpha[gr];
            const int begin = solo ? k0 : k0 + gr;
            for (int k = begin; k < k1; k += 2, ++u) {
                const int buf = u & 1;
                const uint32_t colS = base + (gr * 2 + buf) * 32;
                wait_phase(fd, &ms->s_full[gr][buf], (u >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                const bool masked = key0 + (k + 1) * kTcKeys > ctx;
                const uint32_t sees = masked ? rows_that_see(pi, key0 + k * kTcKeys + t, a.G, a.bt.n) : 0xFFFFFFFFu;
                // the group's previous product has read the weights and written the output
                if (u > 0) wait_phase(fd, &ms->p_done[gr], (u - 1) & 1);
                __syncwarp();
                tc_fence_after();
                // The scores less their maxima (step 0); where one passes 2^8, and on the group's first tile, the scores as they are
                // for new maxima (1), then less those (2).  One copy of the code serves all three.
                float x[NR];
#pragma unroll 1
                for (int step = k > begin ? 0 : 1; step < 3; ++step) {
                    {
                        const float *less = step == 1 ? ms->zero : shift;
                        uint32_t raw[32];
                        tmem_ld32(colS, raw);
                        tc_wait_ld();
#pragma unroll
                        for (int r = 0; r < NR; r += 4) {
                            const float4 m = *reinterpret_cast<const float4 *>(less + r);
                            f2_unpack(f2_fma(f2_from_u32x2(raw[r], raw[r + 1]), c2, f2_pack(m.x, m.y)), x[r], x[r + 1]);
                            f2_unpack(f2_fma(f2_from_u32x2(raw[r + 2], raw[r + 3]), c2, f2_pack(m.z, m.w)), x[r + 2], x[r + 3]);
                        }
                        if (masked) {
#pragma unroll
                            for (int r = 0; r < NR; ++r)
                                if (!((sees >> r) & 1u)) x[r] = -INFINITY;
                        }
                    }
                    if (step == 2) break;
                    if (step == 0) {
                        float over = x[0];
#pragma unroll
                        for (int r = 1; r < NR; ++r) over = fmaxf(over, x[r]);
                        uint32_t grow;
                        asm volatile(
                            "{\n\t.reg .pred p, q;\n\tsetp.gt.f32 p, %1, 0f41000000;\n\t"
                            "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                            : "=r"(grow)
                            : "f"(over), "r"(1 + gr)
                            : "memory");
                        if (!grow) break;
                        continue;
                    }
                    ms->top[gr][wl][lane] = reduce_rows(x, lane, [](float p, float q) { return fmaxf(p, q); });
                    group_sync();
                    if (wl == 0) {
                        const float old = k > begin ? -shift[lane] : kNoMax;
                        const float now = fmaxf(fmaxf(fmaxf(ms->top[gr][0][lane], ms->top[gr][1][lane]), old),
                                                fmaxf(ms->top[gr][2][lane], ms->top[gr][3][lane]));
                        alpha[lane] = ex2_fast(old - now);
                        shift[lane] = -now;
                    }
                    group_sync();
                    if (k > begin) {
#pragma unroll
                        for (int r = 0; r < NR / 2; ++r) l[r] = f2_mul(l[r], *reinterpret_cast<const f32x2 *>(alpha + 2 * r));
#pragma unroll 1
                        for (int j = 0; j < 64; j += 16) {
                            uint32_t o[16];
                            tmem_ld16(colO + j, o);
                            tc_wait_ld();
#pragma unroll
                            for (int r = 0; r < 16; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[(j & 16) + r]);
                            tmem_st16(colO + j, o);
                        }
                        tc_wait_st();
                    }
                }
#pragma unroll
                for (int q = 0; q < NR / 8; ++q) {   // eight rows: one 16-byte chunk of high parts and one of low parts
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = q * 8 + j * 2;
                        const f32x2 e = f2_ex2(f2_pack(x[r], x[r + 1]));
                        l[r / 2] = f2_add(l[r / 2], e);
                        weight_parts(e, hi[j], lo[j]);
                    }
                    sts128(prow + ((q ^ (t & 7)) << 4), hi);
                    sts128(prow + (((q + 4) ^ (t & 7)) << 4), lo);
                }
                if (masked) {
                    // Values that are not finite are replaced by zeros; they are added here for the rows that see them, with the
                    // weights that the product would have used.
                    const uint32_t vs = pi->seq + 2 * (k - k0) + 1, stage = vs % S::STAGES;
                    wait_phase(fd, &fd->kv_full[stage], (vs / S::STAGES) & 1);
                    __syncwarp();
                    scan_values<DP>(sbase + S::OFF_KV + stage * S::TILE, t, fd->vflag[stage]);
                    group_sync();   // the flags and every token's weights are written
                    uint32_t any = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) any |= *reinterpret_cast<volatile uint32_t *>(&fd->vflag[stage][q]);
                    if (any) {
#pragma unroll 1
                        for (int j = 0; j < 128; ++j) {
                            if (!((*reinterpret_cast<volatile uint32_t *>(&fd->vflag[stage][j >> 5]) >> (j & 31)) & 1u)) continue;
                            const int kk = key0 + k * kTcKeys + j;
                            const uint32_t sees = rows_that_see(pi, kk, a.G, a.bt.n);
                            if (kk >= pi->end) continue;   // flags mean nothing after a wait gave up
                            const int64_t off = slot_offset(a.c, a.bt.page_table + pi->table * a.bt.table_pitch, kk);
                            if (off < 0) continue;
                            const float v = t < a.c.head_dim
                                                ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(a.c.v + off + pi->h * a.c.head_b)[t] << 16)
                                                : 0.0f;
                            const char *pj = smem + S::OFF_P + gr * S::PBUF + j * (4 * NR);
                            uint32_t o[32];
                            tmem_ld32(colO, o);
                            tc_wait_ld();
#pragma unroll
                            for (int r = 0; r < NR; ++r) {
                                const int at = (r & 7) * 2;
                                const uint16_t ph = *reinterpret_cast<const uint16_t *>(pj + (((r >> 3) ^ (j & 7)) << 4) + at);
                                const uint16_t pl = *reinterpret_cast<const uint16_t *>(pj + ((((r >> 3) + 4) ^ (j & 7)) << 4) + at);
                                const float w = __uint_as_float((uint32_t)ph << 16) + __uint_as_float((uint32_t)pl << 16);
                                if ((sees >> r) & 1u) o[r] = __float_as_uint(__uint_as_float(o[r]) + w * v);
                            }
                            tmem_st32(colO, o);
                            tc_wait_st();
                        }
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms->p_full[gr]);
            }
            // ---- the piece's end: thread t has head element t
            const int vr = pi->vr, D = a.c.head_dim, qh0 = pi->h * a.G, r0 = pi->r0;
            const bool whole = pi->whole;
            const int ga = solo ? gr : 0;                      // the group that works on it, or the first of the two
            const int bar = solo ? 1 + gr : 3, threads = solo ? 128 : 256;
            auto end_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory"); };
            const size_t slot = (size_t)pi->slot;
            {
                float x[NR];
#pragma unroll
                for (int r = 0; r < NR; r += 2) f2_unpack(l[r / 2], x[r], x[r + 1]);
                ms->top[gr][wl][lane] = reduce_rows(x, lane, [](float p, float q) { return p + q; });
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
            end_sync();
            if (warp == ga * 4) {
                auto sum_of = [&](int g) { return (ms->top[g][0][lane] + ms->top[g][1][lane]) + (ms->top[g][2][lane] + ms->top[g][3][lane]); };
                float m = -ms->shift[ga][lane], f0 = 1.0f, f1 = 0.0f, all = sum_of(ga);
                if (!solo) {
                    const float top0 = m, top1 = -ms->shift[1][lane];
                    m = fmaxf(top0, top1);
                    f0 = ex2_fast(top0 - m);
                    f1 = ex2_fast(top1 - m);
                    all = all * f0 + sum_of(1) * f1;
                }
                const float inv = whole ? (all > 0.0f || all != all ? 1.0f / all : 0.0f) : 1.0f;
                ms->alpha[ga][lane] = f0 * inv;
                if (!solo) ms->alpha[1][lane] = f1 * inv;
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
            // Four rows at a time, the groups taking turns.  Rolled: a piece of one tile goes through all of this once, and the
            // instructions come from far.
#pragma unroll 1
            for (int rb = solo ? 0 : gr * 4; rb < vr; rb += solo ? 4 : 8) {
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
                for (int g = ga; g < (solo ? ga + 1 : 2); ++g) {
                    uint32_t o[4], o2[4];   // the products with the weights' high and low parts
                    tmem_ld4(base + 128 + g * 64 + rb, o);
                    tmem_ld4(base + 128 + g * 64 + 32 + rb, o2);
                    tc_wait_ld();
                    const float4 f = *reinterpret_cast<const float4 *>(ms->alpha[g] + rb);
                    y[0] = fmaf(__uint_as_float(o[0]) + __uint_as_float(o2[0]), f.x, y[0]);
                    y[1] = fmaf(__uint_as_float(o[1]) + __uint_as_float(o2[1]), f.y, y[1]);
                    y[2] = fmaf(__uint_as_float(o[2]) + __uint_as_float(o2[2]), f.z, y[2]);
                    y[3] = fmaf(__uint_as_float(o[3]) + __uint_as_float(o2[3]), f.w, y[3]);
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
        regs_dec<kRegsOther>();
        feed_produce<DP, S::STAGES, NR>(a, a2, fd, sbase, sbase + S::OFF_KV, warp - 8, lane);
    } else {
        regs_dec<kRegsOther>();
        if (warp == 12) {   // the whole warp runs this, with uniform values
            // ------------------------------------------------------------ matrix products
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            constexpr uint32_t shape_o = mma_shape(2 * NR, true, true, false, false);
            uint32_t seq = 0, tiles0 = 0, tiles1 = 0;
            int rests = 0;   // as in the softmax
            // O^T += V^T P^T of the tile whose scores were issued before the last
            int late = 0, late_gr = 0, late_rows = 0;
            uint32_t late_seq = 0, late_u = 0;
            auto weigh = [&]() {
                const uint32_t stage = late_seq % S::STAGES;
                wait_phase(fd, &fd->kv_full[stage], (late_seq / S::STAGES) & 1);
                wait_phase(fd, &ms->p_full[late_gr], late_u & 1);
                __syncwarp();
                if (late_rows) fence_async_smem();
                tc_fence_after();
                const uint64_t v = smem_operand(sbase + S::OFF_KV + stage * S::TILE, DP == 128 ? S::HALF : 0, 1024);
                const uint64_t p = smem_operand(sbase + S::OFF_P + late_gr * S::PBUF, 0, 1024);
                const uint32_t o = tm + 128 + late_gr * 64;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) mma_ss(o, v + kk * (2048 >> 4), p + kk * (2048 >> 4), shape_o, 1u);
                    mma_commit(&fd->kv_empty[stage]);
                    mma_commit(&ms->p_done[late_gr]);
                }
                __syncwarp();
            };
            // Before a wait for what the next scores need: the weighted sum does not wait for it too.
            auto weigh_first = [&](uint64_t *bar, uint32_t parity) {
                if (late && !__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity))) {
                    weigh();
                    late = 0;
                }
            };
            auto ready = [&](uint64_t *bar, uint32_t parity) {
                weigh_first(bar, parity);
                wait_phase(fd, bar, parity);
                __syncwarp();
            };
            for (int it = 0;; ++it) {
                const PieceInfo *pi = &fd->pd[it % kRing];
                weigh_first(&fd->pd_full[it % kRing], (it / kRing) & 1);
                if (!__all_sync(0xFFFFFFFFu, wait_phase<true>(fd, &fd->pd_full[it % kRing], (it / kRing) & 1))) break;
                const int nk = __shfl_sync(0xFFFFFFFFu, pi->k1 - pi->k0, 0);
                if (nk <= 0) break;
                const int rows_from = __shfl_sync(0xFFFFFFFFu, a2.split ? 0 : pi->box_tiles - pi->k0, 0);   // from this tile on, copied by rows
                if (lane == 0) mbar_arrive(&fd->pd_empty[it % kRing]);
                if (nk == 1) rests ^= 1;
                const int first = __shfl_sync(0xFFFFFFFFu, nk == 1 ? rests ^ 1 : 0, 0);   // uniform for the compiler too
                const int qs = it & 1;
                const uint64_t q = smem_operand(sbase + qs * (NR * DP * 2), 16, 1024);
                for (int n = 0; n < nk; ++n) {
                    const int gr = first ^ (n & 1);
                    const uint32_t stage = seq % S::STAGES, u = gr ? tiles1 : tiles0;
                    ready(&fd->kv_full[stage], (seq / S::STAGES) & 1);
                    if (n == 0) {
                        ready(&fd->q_full[qs], (it >> 1) & 1);
                    }
                    if (n == 0 || n >= rows_from) fence_async_smem();
                    tc_fence_after();
                    const uint64_t kt = smem_operand(sbase + S::OFF_KV + stage * S::TILE, 16, 1024);
                    const uint32_t s = tm + (gr * 2 + (u & 1)) * 32;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < DP / 16; ++kk) {
                            const uint32_t ka = ((kk >> 2) * S::HALF + (kk & 3) * 32) >> 4, qa = ((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4;
                            mma_ss(s, kt + ka, q + qa, a2.shape_s, kk > 0);
                        }
                        mma_commit(&ms->s_full[gr][u & 1]);
                        mma_commit(&fd->kv_empty[stage]);
                        if (n == nk - 1) mma_commit(&fd->q_empty[qs]);
                    }
                    __syncwarp();
                    if (late) weigh();
                    late = 1;
                    late_gr = gr;
                    late_rows = n >= rows_from;
                    late_seq = seq + 1;
                    late_u = u;
                    seq += 2;
                    if (gr) ++tiles1;
                    else ++tiles0;
                }
            }
            if (late) weigh();
            if (elect_one()) mma_commit(&ms->done);
            wait_phase<true>(fd, &ms->done, 0);   // the products end by themselves
            __syncwarp();
        } else if (warp == 13) {
            feed_walk(a, a2, fd, ms->walk, lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && fd->dead) feed_drain<S::STAGES>(fd, a.stats);
    if (warp == 12) tmem_free(tmem, 256);
    pdl_wait();   // launched beside the prefixes' kernel: done only when that is, for the join waits for this one
}

template <int DP>
cudaError_t run_few(AttendArgs &a, bool negate, cudaStream_t stream) {
    constexpr size_t bytes = FewShape<DP>::OFF_MISC + sizeof(FewShared);
    static_assert(bytes <= 232448, "shared memory of a block");
    if (prepare_kernel((const void *)k_attend_few<DP>, kTcThreads, bytes) < 1) return cudaErrorInvalidConfiguration;
    const TcArgs t = tc_args(a.c, mma_shape(NR, false, false, false, negate));
    // After the prefixes' kernel of the same call, blocks start as that one's end: they need nothing of it.
    if (a.geo.s0 > 0) return launch_pdl(k_attend_few<DP>, dim3(a.geo.blocks), dim3(kTcThreads), bytes, stream, a, t);
    k_attend_few<DP><<<a.geo.blocks, kTcThreads, bytes, stream>>>(a, t);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_few(AttendArgs &a, cudaStream_t stream) {
    static_assert(kTilesFew.TM == NR && kTilesFew.TK == kTcKeys, "the cutting's tiles are the kernel's");
    a.geo.set(kTilesFew);
    AttendArgs t = a;
    // The maximum is taken after the scale; a negative scale negates the queries in the product, and zero stays zero.
    const bool negate = a.scale_log2 < 0.0f;
    t.scale_log2 = fabsf(a.scale_log2);
    return a.c.head_dim <= 64 ? run_few<64>(t, negate, stream) : run_few<128>(t, negate, stream);
}

}  // namespace sv
