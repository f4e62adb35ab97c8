// sv_attend_few.cuh — what the kernels of sv_kv_attend and sv_kv_attend8 for few packed rows share: the products turned round,
// with tokens along the rows of tensor memory and packed rows along its columns (sv_attend_few.cu says why).
#pragma once

#include "sv_attend_feed.cuh"

namespace sv {

constexpr int NR = kFewRows;
constexpr int kFewReaders = 13;       // warps that read a piece description
constexpr float kNoMax = -1e30f;      // maximum of a row that has seen no token yet

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
    float scale[2];                   // few8: what the groups' outputs are in
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

// The warp that issues the products, run by the whole warp with uniform values.  S: the kernel's shape.  BY_ROWS: tiles may hold rows
// that asynchronous copies wrote, which are fenced here.
template <class S, int DP, bool BY_ROWS>
__device__ __forceinline__ void few_products(Feed *fd, FewShared *ms, const TcArgs &a2, uint32_t sbase, uint32_t tmem, uint32_t shape_o, int lane) {
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
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
        const int rows_from = !BY_ROWS ? INT32_MAX : __shfl_sync(0xFFFFFFFFu, a2.split ? 0 : pi->box_tiles - pi->k0, 0);   // from this tile on, copied by rows
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
}

}  // namespace sv
