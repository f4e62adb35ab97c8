// sv_attend_few32.cu — sv_kv_attend in float32 for up to 8 packed rows a sequence and key head (single tokens and short blocks), heads
// up to 128 wide.
//
// There is next to no arithmetic a byte here (R multiply-adds an element), so each warp works alone, with no block-wide barrier in the
// loop.  It takes 8 tokens of a tile of 64: lanes hold four consecutive elements each, so a token is one coalesced row.  The next
// tile's 8 tokens are copied to shared memory meanwhile.  The 32 scores of 32 / R tokens by R rows are reduced over the lanes together
// (31 shuffles, after which lane j R + r has that of token j and row r), each lane does one exponential, and the weights are handed
// round for the weighted sum.  Warps keep maxima, sums and outputs of their own and are added at the piece's end.
//
// What bounds it: latency of 16 warps an SM, between memory (66% of its peak) and issue slots (51%; 710 instructions a warp and 8
// tokens of 4 rows).  64 sequences of up to 8,192 tokens, 3 key heads of 80, 4 rows: 112 us, 4.6 TB/s or 0.68 of the measured copy
// bandwidth.  With the tiles held in registers instead of copied ahead 176 us, in the kernel for any number of rows 360 us.  One
// thread walks the pieces and leaves them in shared memory: with the walk in every thread's registers 118 us.  The form for 8 rows
// spills 24 bytes.  From width 116 on the ring leaves room for one block an SM, which costs nothing: 8 key heads of 128 take 355 us, 6.2
// TB/s or 0.91 of the copy bandwidth, of 112 (two blocks) 356 us, 5.4 TB/s or 0.79.
#include <type_traits>

#include "sv_attend.cuh"

namespace sv {

namespace {

constexpr int kThreads32 = 256, kWarps32 = 8;

// Sum of x[0..31] over the warp's lanes: lane i gets that of x[i].
__device__ __forceinline__ float sum_lanes(float (&x)[32], int lane) {
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < w) {
                const float mine = up ? x[i + w] : x[i], other = up ? x[i] : x[i + w];
                x[i] = mine + __shfl_xor_sync(0xFFFFFFFFu, other, w);
            }
        }
    }
    return x[0];
}

// Four floats as two packed pairs.
struct Quad {
    f32x2 a, b;
};
__device__ __forceinline__ Quad quad(float4 v) { return {f2_pack(v.x, v.y), f2_pack(v.z, v.w)}; }
__device__ __forceinline__ void scale_quad(Quad &o, float f) {
    const f32x2 f2 = f2_pack(f, f), none = f2_pack(-0.0f, -0.0f);
    o.a = f2_fma(o.a, f2, none);
    o.b = f2_fma(o.b, f2, none);
}

// C8: the cache is held in 8 bits.  Codes are copied as they are, and become floats, times their scale, as they are read.  Issue slots bound that: the
// single tokens above take 128 us (112 over floats, of whose bytes the codes are a quarter; in tiles of 16 rows 403).
template <int R, bool C8>
__global__ void __launch_bounds__(kThreads32, 2) k_attend_few32(const AttendArgs a) {
    constexpr int KB = 32 / R;   // tokens of a batch
    __shared__ Walk s_walk;
    __shared__ Piece s_piece;
    __shared__ bool s_more;
    __shared__ long long warp_sum[kWarps32];
    extern __shared__ __align__(16) float4 ring[];   // [warp][2][8 tokens][keys, values][D / 4]; at a piece's end [warp][R][D / 4]
    __shared__ float s_m[kWarps32][R], s_l[kWarps32][R];
    walk_start<kThreads32>(a, &s_walk, warp_sum);
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    const int D = a.c.head_dim, D4 = D / 4, psize = a.c.page_size;
    const int row = lane % R, slot = lane / R;   // this lane's score of a batch: row, token
    const bool has = lane < D4;                  // the lane holds elements
    float4 *mine = ring + (size_t)wp * 32 * D4;
    const uint32_t mine_at = smem_addr(mine);
    // A tile's 8 tokens are 8 D4 chunks of 16 bytes of keys (of codes a quarter) and as many of values; lane's chunk i is number lane + 32 i.
    constexpr int CHUNKS = C8 ? 2 : 8;
    const int row_chunks = C8 ? D4 / 4 : D4, chunks = 8 * row_chunks;
    int place[CHUNKS];   // token + 8 * (bytes into the row) of the lane's chunks
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
        const int c = lane + 32 * i, j = c / row_chunks;
        place[i] = c < chunks ? j + 8 * 16 * (c - j * row_chunks) : -1;
    }
    const int step_pages = 64 / psize, step_slots = 64 - step_pages * psize;   // a tile further in the page table
    for (int first = 1;; first = 0) {
        if (tid == 0) {
            s_more = s_walk.next(a, s_piece);
            if (first) a.tails[blockIdx.x] = tail_of(a, s_walk, s_piece, s_more);
        }
        __syncthreads();
        if (!s_more) break;
        const Piece p = s_piece;
        const int h = p.h;
        const int32_t *table = a.bt.page_table + p.g.table * a.bt.table_pitch;
        const bool tree = !p.g.chain && p.seg >= a.n_groups;
        Quad q[R], o[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = r / a.G, g = r - i * a.G;   // R covers all rows of a unit
            const char *src = a.q + (int64_t)(p.g.r0 + i) * a.q_row + (int64_t)(h * a.G + g) * a.q_head;
            o[r].a = o[r].b = 0;
            q[r] = r < p.vr && has ? quad(*reinterpret_cast<const float4 *>(src + lane * 16)) : o[r];
        }
        const int my_row = row / a.G;
        const int lim = row >= p.vr ? 0 : p.g.chain ? min(p.g.ctx + my_row + 1, p.end) : tree ? p.g.ctx : p.end;
        uint32_t anc = 0;   // at most 8 rows
        if (tree && row < p.vr) {
            uint32_t words[(SV_MAX_TREE + 32) / 32];
            ancestor_words(a.bt.parents + (int64_t)p.g.table * (a.bt.n - 1), my_row, a.bt.n, words, a.stats, p.g.table);
            anc = words[0];
        }
        float m = -INFINITY, l = 0.0f;
        // Lane j < 8 looks up the warp's token j of the tile after the one that is being copied.
        int next_key = p.g.key0 + p.k0 * 64 + wp * 8 + lane;
        int next_pn = next_key / psize, next_slot = next_key - next_pn * psize, next_page = INT32_MIN;
        auto look_up = [&]() { next_page = lane < 8 && next_key < p.end ? table[next_pn] : INT32_MIN; };
        // C8: scales of the lane's token of the tile at hand, of the next; 1 where that one's page is none of the pool's (not looked at before they are used: a
        // warp stops there until they have come)
        uint32_t kb = 127, vb = 127, kb_next = 127, vb_next = 127;
        bool paged = false;
        auto copy = [&](int k) {   // tile k, which has been looked up; looks up the next
            int64_t off = -1;
            if (C8) {
                paged = (unsigned)next_page < (unsigned)a.c.n_pages;
                const int page = paged ? next_page : 0;
                kb_next = a.sc.k[page * a.sc.page_b + h * a.sc.head_b];
                vb_next = a.sc.v[page * a.sc.page_b + h * a.sc.head_b];
            }
            if (next_page >= 0 && next_page < a.c.n_pages) off = next_page * a.c.page_b + next_slot * a.c.slot_b + h * a.c.head_b;
            else if (next_page != INT32_MIN) report_error(a.stats, SV_ERR_INVALID_ARG, p.g.table);
            next_key += 64;
            next_pn += step_pages;
            next_slot += step_slots;
            if (next_slot >= psize) {
                next_slot -= psize;
                ++next_pn;
            }
            look_up();
            const uint32_t to = mine_at + (uint32_t)((k & 1) * 2 * chunks + lane) * 16;
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                if (32 * i >= chunks) break;
                const int64_t at = __shfl_sync(0xFFFFFFFFu, off, place[i] & 7);
                if (place[i] >= 0) {
                    const int64_t src = at < 0 ? 0 : at + (place[i] >> 3);
                    cp_async16(to + 32 * i * 16, a.c.k + src, at >= 0);
                    cp_async16(to + (32 * i + chunks) * 16, a.c.v + src, at >= 0);
                }
            }
            cp_async_commit();
        };
        look_up();
        copy(p.k0);
        // Where a tile holds hidden tokens, a weight of zero multiplies nothing: their values may not be finite.  Over codes the weights of hidden tokens
        // are -0 and multiply nothing: a NaN reaches every row that sees it, however small the weight.
        auto tile = [&](int k, auto hidden) {
            const int key0 = p.g.key0 + k * 64 + wp * 8;
            const float4 *keys = mine + (k & 1) * 2 * chunks + lane, *values = keys + chunks;
            const uint32_t *kcodes = reinterpret_cast<const uint32_t *>(mine + (k & 1) * 2 * chunks) + lane, *vcodes = kcodes + 4 * chunks;
            // Four elements of the warp's token j: floats, or codes times their scale.
            auto four = [&](const float4 *floats, const uint32_t *codes, float scale, int j) {
                if constexpr (!C8) {
                    return quad(has ? floats[j * D4] : make_float4(0.f, 0.f, 0.f, 0.f));
                } else {
                    Quad x = quad(has ? codes4(codes[j * D4]) : make_float4(0.f, 0.f, 0.f, 0.f));
                    scale_quad(x, scale);
                    return x;
                }
            };
            const float ks = C8 ? scale_of(kb) : 1.0f, vs = C8 ? scale_of(vb) : 1.0f;
#pragma unroll
            for (int b = 0; b < 8 / KB; ++b) {
                float x[32];
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    const Quad kk = four(keys, kcodes, C8 ? __shfl_sync(0xFFFFFFFFu, ks, b * KB + j) : 1.0f, b * KB + j);
#pragma unroll
                    for (int r = 0; r < R; ++r) x[j * R + r] = f2_sum(f2_fma(q[r].a, kk.a, f2_fma(q[r].b, kk.b, 0ull)));
                }
                float s = sum_lanes(x, lane) * a.scale_log2;
                const int key = key0 + b * KB + slot;
                bool sees = true;
                if (hidden.value) {
                    sees = key < lim;
                    if (tree && key >= p.g.ctx && key < p.end) sees = (anc >> (key - p.g.ctx)) & 1u;
                    if (!sees) s = -INFINITY;
                } else if (row >= p.vr) {
                    s = -INFINITY;
                }
                float top = s;
#pragma unroll
                for (int d = R; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                const float now = fmaxf(m, top), ref = now == -INFINITY ? 0.0f : now;
                if (__any_sync(0xFFFFFFFFu, now > m)) {
                    const float alpha = exp2f(m - ref);
                    l *= alpha;
#pragma unroll
                    for (int r = 0; r < R; ++r) scale_quad(o[r], __shfl_sync(0xFFFFFFFFu, alpha, r));
                    m = now;
                }
                const float e = C8 && hidden.value && !sees ? -0.0f : exp2f(s - ref);
                l += e;
#pragma unroll
                for (int j = 0; j < KB; ++j) {
                    const Quad vv = four(values, vcodes, C8 ? __shfl_sync(0xFFFFFFFFu, vs, b * KB + j) : 1.0f, b * KB + j);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float f = __shfl_sync(0xFFFFFFFFu, e, j * R + r);
                        if (!hidden.value || (C8 ? __float_as_uint(f) != 0x80000000u : f != 0.0f)) {
                            const f32x2 f2 = f2_pack(f, f);
                            o[r].a = f2_fma(f2, vv.a, o[r].a);
                            o[r].b = f2_fma(f2, vv.b, o[r].b);
                        }
                    }
                }
            }
        };
        const int seen_by_all = p.seg >= a.n_groups ? p.g.ctx : p.end;
        for (int k = p.k0; k < p.k1; ++k) {
            kb = paged ? kb_next : 127u;
            vb = paged ? vb_next : 127u;
            if (k + 1 < p.k1) {
                copy(k + 1);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            __syncwarp();
            if (p.g.key0 + k * 64 + wp * 8 + 8 <= seen_by_all) tile(k, std::false_type{});
            else tile(k, std::true_type{});
            __syncwarp();   // the half may be overwritten
        }
        // the warps' parts
#pragma unroll
        for (int d = R; d < 32; d <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        if (lane < R) {
            s_m[wp][lane] = m;
            s_l[wp][lane] = l;
        }
        __syncthreads();   // the ring is free
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (has) {
                float4 y;
                f2_unpack(o[r].a, y.x, y.y);
                f2_unpack(o[r].b, y.z, y.w);
                ring[(wp * R + r) * D4 + lane] = y;
            }
        __syncthreads();
        const bool whole = p.k0 == 0 && p.k1 == p.kt && p.seg >= a.n_groups && seg_alone(p.g);
        const size_t at = unit_slot(a, a.geo, p.g, p.seg < a.n_groups, h, p.t) + (size_t)blockIdx.x * a.geo.TM;
        for (int t = tid; t < p.vr * 32; t += kThreads32) {
            const int r = t >> 5, col = t & 31;
            float top = s_m[0][r];
#pragma unroll
            for (int i = 1; i < kWarps32; ++i) top = fmaxf(top, s_m[i][r]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarps32; ++i) {
                const float f = exp2f(s_m[i][r] - ref);
                sum += f * s_l[i][r];
                if (col < D4) {
                    const float4 v = ring[(i * R + r) * D4 + col];
                    y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
                }
            }
            const int i = r / a.G, g = r - i * a.G;
            if (col < D4) {
                if (whole) {
                    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
                    char *dst = a.out + (int64_t)(p.g.r0 + i) * a.o_row + (int64_t)(h * a.G + g) * a.o_head;
                    *reinterpret_cast<float4 *>(dst + col * 16) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
                } else {
                    *reinterpret_cast<float4 *>(a.part + (at + r) * D + col * 4) = y;
                }
            }
            if (col == 0) {
                if (!whole) a.part_ml[at + r] = make_float2(top, sum);
                else if (a.lse)
                    a.lse[(size_t)(p.g.r0 + i) * a.q_heads + h * a.G + g] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
            }
        }
        __syncthreads();
    }
}

template <int R, bool C8>
cudaError_t run_few32(AttendArgs &a, cudaStream_t stream) {
    a.geo.set(tiles_few32(R));
    const size_t bytes = (size_t)kWarps32 * 32 * a.c.head_dim * 4;
    const int resident = prepare_kernel((const void *)k_attend_few32<R, C8>, kThreads32, bytes);
    if (resident < 1) return cudaErrorInvalidConfiguration;
    a.geo.blocks *= resident < 2 ? 1 : 2;
    k_attend_few32<R, C8><<<a.geo.blocks, kThreads32, bytes, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_few32(AttendArgs &a, cudaStream_t stream) {
    if (a.sc.k) return (int64_t)a.bt.n * a.G <= 4 ? run_few32<4, true>(a, stream) : run_few32<8, true>(a, stream);
    return (int64_t)a.bt.n * a.G <= 4 ? run_few32<4, false>(a, stream) : run_few32<8, false>(a, stream);
}

}  // namespace sv
