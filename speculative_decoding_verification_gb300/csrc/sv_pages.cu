// sv_pages.cu — who holds which pages of a cache: new batches from old ones (fork), and the pool's front (compact).
//
// Each call is two kernels.  The plan, one cluster of blocks that meet at hardware barriers, works on the tables and counts: they are
// small (a few entries a thread), so its time is that of its dependent passes (each a load, an atomic or two, a barrier), and one launch takes
// less than one for each pass.  The copy moves whole runs of bytes and is bound by memory; it is launched beside the plan, so that
// its blocks wait where they will run.  In a graph: 256 beams that continue one another, eight layers, 19.3 us (16.5 MB of copies, 2.5 us);
// eight branches of one request 13.6 us; 642 MB moved in eight layers 112 us, 5.7 TB/s, 0.86 of the measured copy bandwidth; a small pool 10.4 us.
#include "sv_kv.cuh"

namespace sv {

namespace {

constexpr int kPlanThreads = 1024, kPlanBlocks = 8;
constexpr int kNobody = INT32_MAX;
constexpr int kPlanMost = 1 << 30;   // pages, and sequences of a new batch: loops step past their ends by less than that

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sum of x over the block's threads before this one; `total` gets all of them.
__device__ __forceinline__ int block_prefix(int x, int *warp_sum, int &total) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += v;
    }
    if (lane == 31) warp_sum[wp] = inc;
    __syncthreads();
    if (wp == 0) {
        int w = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, w, d);
            if (lane >= d) w += v;
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    total = warp_sum[31];
    const int before = inc - x + (wp > 0 ? warp_sum[wp - 1] : 0);
    __syncthreads();
    return before;
}
static_assert(kPlanThreads == 32 * 32, "a warp adds the warps' sums");

// A copy of one page's tokens: to, or -1 for none.
struct PageCopy {
    int32_t from, to, tokens;
};

struct ForkArgs {
    const int32_t *refs, *context_len, *table, *src;
    int64_t pitch, out_pitch;
    int max_pages, B, N, reserve, n_pages, page_size;
    int32_t *refs_out, *table_out, *context_out;
    sv_stats *stats;
    // workspace
    int2 *holders;       // [n_pages] those of the old table (x), and new sequences that share the page (y)
    int32_t *owner;      // [n_pages] first new sequence whose last tokens fill the page in part
    int32_t *free_list;  // [n_pages] free pages, rising
    int32_t *counts;     // [2][kPlanBlocks] free pages and wanted pages of a block's part
    PageCopy *copies;    // [N]
};

struct Child {
    int ctx, full, entries;   // tokens; entries that are shared; entries that name a page (0: the sequence is empty)
    const int32_t *row;       // of the old table
    bool part;                // the last tokens fill a page in part
};

// Sequence j of the new batch, with every device value checked.
__device__ __forceinline__ Child child_of(const ForkArgs &a, int j, bool report) {
    const int b = a.src[j];
    Child c{0, 0, 0, nullptr, false};
    if (b < 0 || b >= a.B) {
        if (report && b != -1) report_error(a.stats, SV_ERR_INVALID_ARG, j);
        return c;
    }
    const int ctx = a.context_len[b];
    if (ctx < 0 || (int64_t)ctx + a.reserve > (int64_t)a.max_pages * a.page_size) {
        if (report) report_error(a.stats, SV_ERR_INVALID_ARG, j);
        return c;
    }
    c.ctx = ctx;
    c.full = ctx / a.page_size;
    c.part = ctx - c.full * a.page_size > 0;
    c.entries = (int)(((int64_t)ctx + a.reserve + a.page_size - 1) / a.page_size);
    c.row = a.table + b * a.pitch;
    return c;
}

__global__ void __cluster_dims__(kPlanBlocks, 1, 1) __launch_bounds__(kPlanThreads, 1) k_fork_plan(const ForkArgs a) {
    __shared__ int warp_sum[32];
    const int tid = threadIdx.x, me = blockIdx.x, all = kPlanBlocks * kPlanThreads;
    const int first = me * kPlanThreads + tid;
    pdl_trigger();
    for (int p = first; p < a.n_pages; p += all) {
        a.holders[p] = make_int2(0, 0);
        a.owner[p] = kNobody;
    }
    cluster_sync();
    // holders that go, holders that come, and who asks for a partly filled page
    for (int64_t e = first; e < (int64_t)a.B * a.max_pages; e += all) {
        const int b = (int)(e / a.max_pages), p = a.table[b * a.pitch + (e - (int64_t)b * a.max_pages)];
        if (p >= a.n_pages) report_error(a.stats, SV_ERR_INVALID_ARG, b);
        else if (p >= 0) atomicAdd(&a.holders[p].x, 1);
    }
    const int warp = first >> 5, warps = all >> 5, lane = tid & 31;
    for (int j = warp; j < a.N; j += warps) {
        const Child c = child_of(a, j, lane == 0);
        const int named = c.full + c.part;   // entries with tokens
        for (int e = lane; e < named; e += 32) {
            const int p = c.row[e];
            if ((unsigned)p >= (unsigned)a.n_pages) report_error(a.stats, SV_ERR_INVALID_ARG, j);
            else if (e < c.full) atomicAdd(&a.holders[p].y, 1);
            else atomicMin(&a.owner[p], j);
        }
    }
    cluster_sync();
    // pages: a block takes a run of them, a thread a run of that
    const int each = (a.n_pages + all - 1) / all;
    const int p0 = min((int64_t)a.n_pages, (int64_t)first * each), p1 = min(a.n_pages, p0 + each);
    int free_here = 0;
    for (int p = p0; p < p1; ++p) {
        // counted apart: a page whose count lacks holders is reported, and is not free while a sequence comes to it
        const int2 held = a.holders[p];
        const int others = a.refs[p] - held.x;
        if (others < 0) report_error(a.stats, SV_ERR_INVALID_ARG, p);
        int r = max(others, 0) + held.y;
        if (a.owner[p] != kNobody) {
            if (r == 0) r = 1;   // the first new sequence keeps it
            else a.owner[p] = kNobody;
        }
        a.refs_out[p] = r;
        free_here += r == 0;
    }
    int total;
    int rank = block_prefix(free_here, warp_sum, total);
    if (tid == 0) a.counts[me] = total;
    cluster_sync();
    int n_free = 0;
    for (int k = 0; k < kPlanBlocks; ++k) {
        const int n = *reinterpret_cast<volatile int32_t *>(&a.counts[k]);
        rank += k < me ? n : 0;
        n_free += n;
    }
    for (int p = p0; p < p1; ++p)
        if (a.refs_out[p] == 0) a.free_list[rank++] = p;
    // sequences: the same split
    const int many = (a.N + all - 1) / all;
    const int j0 = min((int64_t)a.N, (int64_t)first * many), j1 = min(a.N, j0 + many);
    auto keeps = [&](const Child &c, int j) {
        if (!c.part) return false;
        const int p = c.row[c.full];
        return (unsigned)p < (unsigned)a.n_pages && a.owner[p] == j;
    };
    int wants = 0;
    for (int j = j0; j < j1; ++j) {
        const Child c = child_of(a, j, false);
        if (c.entries > 0) wants += c.entries - c.full - keeps(c, j);
    }
    int before = block_prefix(wants, warp_sum, total);
    if (tid == 0) a.counts[kPlanBlocks + me] = total;
    cluster_sync();
    for (int k = 0; k < me; ++k) before += *reinterpret_cast<volatile int32_t *>(&a.counts[kPlanBlocks + k]);
    for (int j = j0; j < j1; ++j) {   // where a sequence's new pages start in the list, for the warp that writes its row
        const Child c = child_of(a, j, false);
        a.copies[j].from = before;
        if (c.entries > 0) before += c.entries - c.full - keeps(c, j);
    }
    cluster_sync();
    for (int j = warp; j < a.N; j += warps) {
        const Child c = child_of(a, j, false);
        const bool kept = keeps(c, j);
        const int from = a.copies[j].from, fresh = c.full + kept;   // entries from here on are given pages
        __syncwarp();
        PageCopy copy{0, -1, 0};
        for (int e = lane; e < a.max_pages; e += 32) {
            int p = -1;
            if (e < fresh) {
                p = (unsigned)c.row[e] < (unsigned)a.n_pages ? c.row[e] : -1;
            } else if (e < c.entries) {
                const int k = from + e - fresh;
                if (k < n_free) {
                    p = a.free_list[k];
                    a.refs_out[p] = 1;
                } else {
                    report_error(a.stats, SV_ERR_NO_PAGE, j);
                }
                if (e == c.full && c.part && p >= 0) {
                    const int old = c.row[e];
                    if ((unsigned)old < (unsigned)a.n_pages) copy = {old, p, c.ctx - c.full * a.page_size};
                }
            }
            a.table_out[j * a.out_pitch + e] = p;
        }
        const uint32_t has = __ballot_sync(0xFFFFFFFFu, copy.to >= 0);
        const int from_lane = has ? __ffs(has) - 1 : 0;
        copy.from = __shfl_sync(0xFFFFFFFFu, copy.from, from_lane);
        copy.to = __shfl_sync(0xFFFFFFFFu, copy.to, from_lane);
        copy.tokens = __shfl_sync(0xFFFFFFFFu, copy.tokens, from_lane);
        if (lane == 0) {
            a.copies[j] = copy;
            a.context_out[j] = c.ctx;
        }
    }
}

// Tokens of a page in one layer as runs of bytes: `outer` by `inner` runs (by head and token, or the other way round), each `run` long.  Where the
// layout lets neighbours touch they are one run.
struct PageRuns {
    char *k, *v;
    uint8_t *k_scale, *v_scale;
    int64_t layer_b, page_b, token_b, head_b, scale_layer_b, scale_page_b, scale_head_b;
    int layers, heads, scale_heads;
    int run;            // bytes a token and (merged) head
    bool tokens_touch;  // the next token's bytes follow: runs of all tokens
};

inline PageRuns page_runs(const sv_kv_pool &p) {
    PageRuns r{static_cast<char *>(p.k), static_cast<char *>(p.v), p.k_scale, p.v_scale, p.layer_stride, p.page_stride, p.slot_stride, p.head_stride,
               p.scale_layer_stride, p.scale_page_stride, p.scale_head_stride, p.n_layers, p.kv_heads, p.kv_heads, (int)p.head_bytes, false};
    if (r.heads == 1 || (p.head_stride == p.head_bytes && p.head_bytes * p.kv_heads <= INT32_MAX / 4)) {
        r.run = (int)(p.head_bytes * p.kv_heads);
        r.heads = 1;
    }
    r.tokens_touch = r.token_b == r.run && (int64_t)r.run * p.page_size <= INT32_MAX / 4;
    return r;
}

// Copies `tokens` tokens of page `from` to page `to` in one layer, by the whole block.  Loads go ahead of their stores, four a thread.
__device__ __forceinline__ void copy_page(const PageRuns &r, int64_t layer, int from, int to, int tokens) {
    const int vecs = (r.tokens_touch ? r.run * tokens : r.run) / 16, toks = r.tokens_touch ? 1 : tokens;
    const int per_head = vecs * toks, all = 2 * r.heads * per_head;
    const int64_t base = layer * r.layer_b, step = (int64_t)(to - from) * r.page_b;
    auto place = [&](int u) {
        const int which = u >= r.heads * per_head;
        u -= which * r.heads * per_head;
        const int h = r.heads == 1 ? 0 : u / per_head;
        u -= h * per_head;
        const int t = toks == 1 ? 0 : u / vecs;
        return (which ? r.v : r.k) + base + from * r.page_b + h * r.head_b + t * r.token_b + (u - t * vecs) * 16;
    };
    for (int u0 = threadIdx.x; u0 < all; u0 += 4 * blockDim.x) {
        char *at[4];
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = u0 + i * blockDim.x;
            if (u < all) {
                at[i] = place(u);
                w[i] = *reinterpret_cast<const uint4 *>(at[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (u0 + i * (int)blockDim.x < all) *reinterpret_cast<uint4 *>(at[i] + step) = w[i];
    }
    if (r.k_scale != nullptr) {
        for (int u = threadIdx.x; u < 2 * r.scale_heads; u += blockDim.x) {
            const int which = u >= r.scale_heads;
            uint8_t *s = (which ? r.v_scale : r.k_scale) + layer * r.scale_layer_b + (u - which * r.scale_heads) * r.scale_head_b;
            s[to * r.scale_page_b] = s[from * r.scale_page_b];
        }
    }
}

__global__ void __launch_bounds__(256) k_fork_copy(const PageRuns r, const PageCopy *copies, int N) {
    pdl_wait();
    const int j = blockIdx.x % N;
    const PageCopy c = copies[j];
    if (c.to >= 0) copy_page(r, blockIdx.x / N, c.from, c.to, c.tokens);
}

struct CompactArgs {
    const int32_t *refs, *table;
    int64_t pitch, out_pitch;
    int max_pages, B, n_pages;
    int32_t *refs_out, *table_out, *moved_to, *live;
    sv_stats *stats;
    // workspace
    int32_t *to;       // [n_pages] new number
    int32_t *from;     // [n_pages] of the k-th move
    int32_t *hole;     // [n_pages]
    int32_t *counts;   // [2][kPlanBlocks]
    int32_t *moves;    // [1]
};

__global__ void __cluster_dims__(kPlanBlocks, 1, 1) __launch_bounds__(kPlanThreads, 1) k_compact_plan(const CompactArgs a) {
    __shared__ int warp_sum[32];
    const int tid = threadIdx.x, me = blockIdx.x, all = kPlanBlocks * kPlanThreads;
    const int first = me * kPlanThreads + tid;
    pdl_trigger();
    const int each = (a.n_pages + all - 1) / all;
    const int p0 = min((int64_t)a.n_pages, (int64_t)first * each), p1 = min(a.n_pages, p0 + each);
    int n = 0, total;
    for (int p = p0; p < p1; ++p) {
        const int r = a.refs[p];
        if (r < 0) report_error(a.stats, SV_ERR_INVALID_ARG, p);
        n += r > 0;
    }
    const int held_before = block_prefix(n, warp_sum, total);
    if (tid == 0) a.counts[me] = total;
    cluster_sync();
    int rank = held_before, live = 0;   // pages held before p0
    for (int k = 0; k < kPlanBlocks; ++k) {
        const int c = *reinterpret_cast<volatile int32_t *>(&a.counts[k]);
        rank += k < me ? c : 0;
        live += c;
    }
    // The k-th hole below L, and the k-th page at or above L, count those before them: before page p there are p - rank holes and, from
    // L on, rank - (pages held below L) pages to move.  As many are held below L as there are not holes there.
    int below = 0;   // holes below L in this thread's part
    {
        int k = rank;
        for (int p = p0; p < p1; ++p) {
            const bool held = a.refs[p] > 0;
            if (!held && p < live) {
                a.hole[p - k] = p;
                ++below;
            }
            k += held;
        }
    }
    block_prefix(below, warp_sum, total);
    if (tid == 0) a.counts[kPlanBlocks + me] = total;
    cluster_sync();
    int holes = 0;
    for (int k = 0; k < kPlanBlocks; ++k) holes += *reinterpret_cast<volatile int32_t *>(&a.counts[kPlanBlocks + k]);
    const int held_below = live - holes;
    for (int p = p0; p < p1; ++p) {
        const int r = a.refs[p];
        int to = -1;
        if (r > 0) {
            to = p;
            if (p >= live) {
                const int k = rank - held_below;
                to = a.hole[k];
                a.from[k] = p;
            }
            ++rank;
        }
        a.to[p] = to;
        if (a.moved_to) a.moved_to[p] = to;
    }
    if (first == 0) {
        a.live[0] = live;
        a.moves[0] = holes;
    }
    cluster_sync();
    // Counts move with their pages.  In place, a page's own count is read before the loop that clears it.
    for (int k = first; k < holes; k += all) a.refs_out[a.hole[k]] = a.refs[a.from[k]];
    cluster_sync();
    for (int p = first; p < a.n_pages; p += all) {
        if (p >= live) a.refs_out[p] = 0;
        else if (a.to[p] == p) a.refs_out[p] = a.refs[p];
    }
    for (int64_t e = first; e < (int64_t)a.B * a.max_pages; e += all) {
        const int b = (int)(e / a.max_pages), c = (int)(e - (int64_t)b * a.max_pages), p = a.table[b * a.pitch + c];
        int to = p;
        if (p >= 0) {
            to = p < a.n_pages ? a.to[p] : -1;
            if (to < 0) {
                report_error(a.stats, SV_ERR_INVALID_ARG, b);
                to = p;
            }
        }
        a.table_out[b * a.out_pitch + c] = to;
    }
}

__global__ void __launch_bounds__(256) k_compact_copy(const PageRuns r, const int32_t *from, const int32_t *hole, const int32_t *moves, int page_size) {
    pdl_wait();
    const int64_t all = (int64_t)*moves * r.layers;
    for (int64_t u = blockIdx.x; u < all; u += gridDim.x) {
        const int64_t layer = u % r.layers;
        const int k = (int)(u / r.layers);
        copy_page(r, layer, from[k], hole[k], page_size);
    }
}

bool pool_ok(const sv_kv_pool *p) {
    if (p == nullptr || p->k == nullptr || p->v == nullptr || (p->k_scale == nullptr) != (p->v_scale == nullptr)) return false;
    if (p->n_layers < 1 || p->n_pages < 1 || p->n_pages > kPlanMost || p->page_size < 1 || p->kv_heads < 1 || p->head_bytes < 1 || p->head_bytes > 4 * SV_KV_MAX_HEAD_DIM)
        return false;
    // offsets of a page's vectors are formed in 32 bits
    if ((int64_t)p->page_size * p->kv_heads > INT32_MAX || (int64_t)p->page_size * p->kv_heads * (p->head_bytes / 16) > INT32_MAX / 8) return false;
    return aligned(p->k, 16) && aligned(p->v, 16) && p->layer_stride % 16 == 0 && p->page_stride % 16 == 0 && p->slot_stride % 16 == 0 &&
           p->head_stride % 16 == 0 && p->head_bytes % 16 == 0;
}

// Whether [a, a + n) and [b, b + m) int32 elements share some.
bool share(const int32_t *a, int64_t n, const int32_t *b, int64_t m) {
    return a != nullptr && b != nullptr && n > 0 && m > 0 && (uintptr_t)a < (uintptr_t)(b + m) && (uintptr_t)b < (uintptr_t)(a + n);
}
int64_t table_extent(int rows, int64_t pitch, int width) { return rows > 0 ? (rows - 1) * pitch + width : 0; }

struct ForkPlan {
    size_t holders, owner, list, counts, copies, bytes;
};
ForkPlan plan_fork(int n_pages, int N) {
    Carver cv;
    ForkPlan p{};
    p.holders = cv.take<int2>(n_pages);
    p.owner = cv.take<int32_t>(n_pages);
    p.list = cv.take<int32_t>(n_pages);
    p.counts = cv.take<int32_t>(2 * kPlanBlocks);
    p.copies = cv.take<PageCopy>(N);
    p.bytes = cv.off + 256;
    return p;
}
struct CompactPlan {
    size_t to, from, hole, counts, moves, bytes;
};
CompactPlan plan_compact(int n_pages) {
    Carver cv;
    CompactPlan p{};
    p.to = cv.take<int32_t>(n_pages);
    p.from = cv.take<int32_t>(n_pages);
    p.hole = cv.take<int32_t>(n_pages);
    p.counts = cv.take<int32_t>(2 * kPlanBlocks);
    p.moves = cv.take<int32_t>(1);
    p.bytes = cv.off + 256;
    return p;
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" size_t sv_kv_fork_workspace_size(int n_pages, int N) { return n_pages < 1 || N < 1 ? 0 : plan_fork(n_pages, N).bytes; }

extern "C" sv_status sv_kv_fork(const sv_kv_pool *pool, const int32_t *refs, const int32_t *context_len, const int32_t *page_table,
                                int64_t table_pitch, int max_pages, int B, const int32_t *src, int N, int reserve,
                                int32_t *refs_out, int32_t *table_out, int64_t table_out_pitch, int32_t *context_out,
                                sv_stats *stats, void *workspace, size_t workspace_bytes, sv_stream_t stream) {
    if (!pool_ok(pool) || refs == nullptr || context_len == nullptr || page_table == nullptr || src == nullptr || refs_out == nullptr ||
        table_out == nullptr || context_out == nullptr || B < 1 || N < 1 || max_pages < 1 || reserve < 0 || table_pitch < max_pages ||
        table_out_pitch < max_pages)
        return SV_ERR_INVALID_ARG;
    if ((int64_t)max_pages * pool->page_size > kMaxSlots || (int64_t)B * max_pages > INT32_MAX || (int64_t)N * max_pages > INT32_MAX ||
        (int64_t)N * pool->n_layers > INT32_MAX || N > kPlanMost)
        return SV_ERR_INVALID_ARG;
    const int n_pages = pool->n_pages;
    const int64_t in = table_extent(B, table_pitch, max_pages), out = table_extent(N, table_out_pitch, max_pages);
    if (refs_out != refs && share(refs, n_pages, refs_out, n_pages)) return SV_ERR_INVALID_ARG;
    const struct {
        const int32_t *p;
        int64_t n;
    } ins[] = {{refs, n_pages}, {context_len, B}, {page_table, in}, {src, N}}, outs[] = {{refs_out, n_pages}, {table_out, out}, {context_out, N}};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 4; ++i)
            if ((o > 0 || i > 0) && share(ins[i].p, ins[i].n, outs[o].p, outs[o].n)) return SV_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i)
            if (share(outs[i].p, outs[i].n, outs[o].p, outs[o].n)) return SV_ERR_INVALID_ARG;
    }
    const ForkPlan pl = plan_fork(n_pages, N);
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < pl.bytes) return SV_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on_current_device(s, pool->k, refs)) return SV_ERR_INVALID_ARG;
    if (stats && cudaMemsetAsync(stats, 0, sizeof(sv_stats), s) != cudaSuccess) return SV_ERR_CUDA;
    char *w = static_cast<char *>(workspace);
    ForkArgs a{refs, context_len, page_table, src, table_pitch, table_out_pitch, max_pages, B, N, reserve, n_pages, pool->page_size,
               refs_out, table_out, context_out, stats};
    a.holders = reinterpret_cast<int2 *>(w + pl.holders);
    a.owner = reinterpret_cast<int32_t *>(w + pl.owner);
    a.free_list = reinterpret_cast<int32_t *>(w + pl.list);
    a.counts = reinterpret_cast<int32_t *>(w + pl.counts);
    a.copies = reinterpret_cast<PageCopy *>(w + pl.copies);
    k_fork_plan<<<kPlanBlocks, kPlanThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = launch_pdl(k_fork_copy, dim3((unsigned)((int64_t)N * pool->n_layers)), dim3(256), 0, s, page_runs(*pool), a.copies, N);
    return cuda_status(e);
}

extern "C" size_t sv_kv_compact_workspace_size(int n_pages) { return n_pages < 1 ? 0 : plan_compact(n_pages).bytes; }

extern "C" sv_status sv_kv_compact(const sv_kv_pool *pool, const int32_t *refs, const int32_t *page_table, int64_t table_pitch,
                                   int max_pages, int B, int32_t *refs_out, int32_t *table_out, int64_t table_out_pitch,
                                   int32_t *moved_to, int32_t *live, sv_stats *stats, void *workspace, size_t workspace_bytes,
                                   sv_stream_t stream) {
    if (!pool_ok(pool) || refs == nullptr || refs_out == nullptr || live == nullptr || B < 0) return SV_ERR_INVALID_ARG;
    if (B > 0 && (page_table == nullptr || table_out == nullptr || max_pages < 1 || table_pitch < max_pages || table_out_pitch < max_pages ||
                  (int64_t)B * max_pages > INT32_MAX || (table_out == page_table && table_out_pitch != table_pitch)))
        return SV_ERR_INVALID_ARG;
    const int n_pages = pool->n_pages;
    const int64_t in = table_extent(B, table_pitch, max_pages), out = table_extent(B, table_out_pitch, max_pages);
    if ((refs_out != refs && share(refs, n_pages, refs_out, n_pages)) || (table_out != page_table && share(page_table, in, table_out, out)))
        return SV_ERR_INVALID_ARG;
    const struct {
        const int32_t *p;
        int64_t n;
    } outs[] = {{refs_out, n_pages}, {table_out, out}, {moved_to, n_pages}, {live, 1}};
    for (int o = 0; o < 4; ++o) {
        if ((o != 0 && share(refs, n_pages, outs[o].p, outs[o].n)) || (o != 1 && share(page_table, in, outs[o].p, outs[o].n)))
            return SV_ERR_INVALID_ARG;
        for (int i = 0; i < o; ++i)
            if (share(outs[i].p, outs[i].n, outs[o].p, outs[o].n)) return SV_ERR_INVALID_ARG;
    }
    const CompactPlan pl = plan_compact(n_pages);
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < pl.bytes) return SV_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    DeviceInfo di;
    if (!on_current_device(s, pool->k, refs)) return SV_ERR_INVALID_ARG;
    if (!device_info(di)) return SV_ERR_CUDA;
    if (stats && cudaMemsetAsync(stats, 0, sizeof(sv_stats), s) != cudaSuccess) return SV_ERR_CUDA;
    char *w = static_cast<char *>(workspace);
    CompactArgs a{refs, page_table, table_pitch, table_out_pitch, max_pages, B, n_pages, refs_out, table_out, moved_to, live, stats};
    a.to = reinterpret_cast<int32_t *>(w + pl.to);
    a.from = reinterpret_cast<int32_t *>(w + pl.from);
    a.hole = reinterpret_cast<int32_t *>(w + pl.hole);
    a.counts = reinterpret_cast<int32_t *>(w + pl.counts);
    a.moves = reinterpret_cast<int32_t *>(w + pl.moves);
    k_compact_plan<<<kPlanBlocks, kPlanThreads, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    const int64_t most = ((int64_t)n_pages / 2 + 1) * pool->n_layers, resident = (int64_t)di.sms * 8;   // at most half of the pages move
    if (e == cudaSuccess)
        e = launch_pdl(k_compact_copy, dim3((unsigned)(most < resident ? most : resident)), dim3(256), 0, s, page_runs(*pool),
                       (const int32_t *)a.from, (const int32_t *)a.hole, (const int32_t *)a.moves, pool->page_size);
    return cuda_status(e);
}
