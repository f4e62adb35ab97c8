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
    alignas(16) float alpha[2][NR];   // what a new maximum scales the row by; at the end what the group's output is scaled by
};

// Whether a weighted sum has to be issued before anything else, by a warp that issues scores up to three tiles ahead of them.  `waiting` tiles have
// scores and no sum yet; `groups` has their groups, a bit each; `next` is the group whose scores come next, or -1.  A group has two score
// buffers, and the softmax has read one for good when it has written the tile's weights, which the tile's sum waits for: with two tiles of the
// group waiting, the next tile's scores would go over ones that are still read.  Groups take turns within a piece, but a piece of one tile goes to either: an
// odd number of tiles, a piece of one and the next piece's first can be three of one group in a row.
SV_HD bool sum_is_due(uint32_t waiting, uint32_t groups, int next) {
    return waiting == 3 || (waiting == 2 && next >= 0 && groups == (next ? 3u : 0u));
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

}  // namespace sv
