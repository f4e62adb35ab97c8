// sv_attend.cu — sv_kv_attend: the float32-arithmetic kernel, the join of partial results, the entry point.
#include <math.h>
#include <type_traits>

#include "sv_attend.cuh"

namespace sv {

constexpr int kAttThreads = 256;

// Four consecutive elements in shared memory, as float32.
template <int ES>
__device__ __forceinline__ float4 lds4(const char *p) {
    if constexpr (ES == 4) {
        return *reinterpret_cast<const float4 *>(p);
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
    }
}

template <int ES, int DP, int TM>
struct F32Shape {
    static constexpr int TK = DP == 256 ? 32 : 64;
    static constexpr int RG = TM / 4;                       // groups of four rows
    static constexpr int TPR = kAttThreads / RG;            // threads of a row group
    static constexpr int NK = TK >= TPR ? TK / TPR : 1;     // keys a thread scores
    static constexpr int CG = DP / 4;                       // groups of four columns
    static constexpr int KS = TPR > CG ? TPR / CG : 1;      // keys split over threads in the weighted sum
    static constexpr int NC = TPR > CG ? 1 : CG / TPR;      // column groups of a thread
    static constexpr int ROW = DP * ES + 16;                // bytes of a key row, padded off the banks
    static constexpr int SP = TK + 4;                       // floats of a score row
    static constexpr int ANC = (SV_MAX_TREE + 32) / 32;
    static constexpr size_t OFF_K = (size_t)TM * DP * 4;
    static constexpr size_t OFF_V = OFF_K + 2 * (size_t)TK * ROW;
    static constexpr size_t OFF_S = OFF_V + 2 * (size_t)TK * ROW;
    static constexpr size_t OFF_M = OFF_S + (size_t)TM * SP * 4;
    static constexpr size_t BYTES = OFF_M + (size_t)TM * 4 * (4 + ANC) + 64;
};

// Scores, softmax and weighted sum in float32 FMA, a tile of TM packed rows by TK keys at a time.  Threads hold
// 4 rows by NK keys of the scores and 4 rows by 4 NC columns of the output; keys and values are
// double buffered with asynchronous copies.  For float32 with more rows than few32 takes and for bf16 heads wider than 128: the
// FMA rate and, with few rows, the four block barriers a tile bound it.
template <int ES, int DP, int TM>
__global__ void __launch_bounds__(kAttThreads) k_attend_f32(const AttendArgs a) {
    using S = F32Shape<ES, DP, TM>;
    constexpr int TK = S::TK;
    extern __shared__ __align__(128) char smem[];
    __shared__ Walk s_walk;
    __shared__ long long warp_sum[kAttThreads / 32];
    float *sq = reinterpret_cast<float *>(smem);
    char *sk = smem + S::OFF_K, *sv_ = smem + S::OFF_V;
    float *ss = reinterpret_cast<float *>(smem + S::OFF_S);
    float *row_m = reinterpret_cast<float *>(smem + S::OFF_M), *row_l = row_m + TM, *row_a = row_l + TM;
    int *row_lim = reinterpret_cast<int *>(row_a + TM);
    uint32_t *row_anc = reinterpret_cast<uint32_t *>(row_lim + TM);

    walk_start<kAttThreads>(a, &s_walk, warp_sum);
    pdl_trigger();
    Walk w = s_walk;
    const int tid = threadIdx.x, lane = tid & 31, wp = tid >> 5;
    const int D = a.c.head_dim, D4 = D / 4, chunks = D * ES / 16;
    const int rg = tid / S::TPR, tx = tid % S::TPR;
    const int cx = tx % S::CG, ks = S::KS > 1 ? tx / S::CG : 0;
    Piece p;
    for (int first = 1;; first = 0) {
        const bool more = w.next(a, p);
        if (first && tid == 0) a.tails[blockIdx.x] = tail_of(a, w, p, more);
        if (!more) break;
        const int m0 = p.t * TM, h = p.h;
        const int32_t *table = a.bt.page_table + p.g.table * a.bt.table_pitch;
        auto load_tile = [&](int k, int buf) {
            const int first = p.g.key0 + k * TK + wp * (TK / 8);
            int64_t off = -1;
            if (lane < TK / 8 && first + lane < p.end) {
                off = slot_offset(a.c, table, first + lane);
                if (off < 0) report_error(a.stats, SV_ERR_INVALID_ARG, p.g.table);
            }
#pragma unroll
            for (int r = 0; r < TK / 8; ++r) {
                const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
                const size_t dst = (size_t)(buf * TK + wp * (TK / 8) + r) * S::ROW;
                for (int c = lane; c < chunks; c += 32) {
                    const int64_t src = o < 0 ? 0 : o + h * a.c.head_b + c * 16;
                    cp_async16(smem_addr(sk + dst + c * 16), a.c.k + src, o >= 0);
                    cp_async16(smem_addr(sv_ + dst + c * 16), a.c.v + src, o >= 0);
                }
            }
            cp_async_commit();
        };
        load_tile(p.k0, 0);
        for (int i = tid; i < TM * D4; i += kAttThreads) {
            const int m = i / D4, d = i - m * D4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (m < p.vr) {
                const int r = (m0 + m) / a.G, g = m0 + m - r * a.G;
                const char *src = a.q + (int64_t)(p.g.r0 + r) * a.q_row + (int64_t)(h * a.G + g) * a.q_head + d * 4 * ES;
                x = lds4<ES>(src);
            }
            *reinterpret_cast<float4 *>(sq + m * DP + d * 4) = x;
        }
        const bool tree = !p.g.chain && p.seg >= a.n_groups;
        if (tid < TM) {
            const int i = (m0 + tid) / a.G;
            row_m[tid] = -INFINITY;
            row_l[tid] = 0.0f;
            row_lim[tid] = tid >= p.vr ? 0 : p.g.chain ? min(p.g.ctx + i + 1, p.end) : tree ? p.g.ctx : p.end;
            if (tree) {
                uint32_t anc[S::ANC] = {};
                if (tid < p.vr) ancestor_words(a.bt.parents + (int64_t)p.g.table * (a.bt.n - 1), i, a.bt.n, anc, a.stats, p.g.table);
#pragma unroll
                for (int j = 0; j < S::ANC; ++j) row_anc[tid * S::ANC + j] = anc[j];
            }
        }
        float4 acc[4][S::NC];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < S::NC; ++c) acc[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);

        for (int k = p.k0; k < p.k1; ++k) {
            const int buf = (k - p.k0) & 1;
            if (k + 1 < p.k1) {
                load_tile(k + 1, buf ^ 1);
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
            __syncthreads();
            const char *tk = sk + (size_t)buf * TK * S::ROW, *tv = sv_ + (size_t)buf * TK * S::ROW;
            const int first = p.g.key0 + k * TK;
            if (tx < TK) {
                float s[4][S::NK] = {};
                for (int d = 0; d < D4; ++d) {
                    float4 qv[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) qv[r] = *reinterpret_cast<const float4 *>(sq + (rg * 4 + r) * DP + d * 4);
#pragma unroll
                    for (int j = 0; j < S::NK; ++j) {
                        const float4 kv = lds4<ES>(tk + (size_t)(tx + j * S::TPR) * S::ROW + d * 4 * ES);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            s[r][j] = fmaf(qv[r].x, kv.x, fmaf(qv[r].y, kv.y, fmaf(qv[r].z, kv.z, fmaf(qv[r].w, kv.w, s[r][j]))));
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < S::NK; ++j) ss[(rg * 4 + r) * S::SP + tx + j * S::TPR] = s[r][j] * a.scale_log2;
            }
            __syncthreads();
            // softmax: a warp takes rows wp, wp + 8, ...
            for (int m = wp; m < TM; m += 8) {
                const int lim = row_lim[m];
                float x[TK / 32], top = -INFINITY;
#pragma unroll
                for (int j = 0; j < TK / 32; ++j) {
                    const int key = first + lane + j * 32;
                    bool sees = key < lim;
                    if (tree && m < p.vr && key >= p.g.ctx && key < p.end) {
                        const int rel = key - p.g.ctx;
                        sees = (row_anc[m * S::ANC + (rel >> 5)] >> (rel & 31)) & 1u;
                    }
                    x[j] = sees ? ss[m * S::SP + lane + j * 32] : -INFINITY;
                    top = fmaxf(top, x[j]);
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                const float m_old = row_m[m], m_new = fmaxf(m_old, top);
                const float base = m_new == -INFINITY ? 0.0f : m_new;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < TK / 32; ++j) {
                    const float e = exp2f(x[j] - base);
                    ss[m * S::SP + lane + j * 32] = e;
                    sum += e;
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
                __syncwarp();
                if (lane == 0) {
                    const float alpha = exp2f(m_old - base);
                    row_a[m] = alpha;
                    row_m[m] = m_new;
                    row_l[m] = row_l[m] * alpha + sum;
                }
            }
            __syncthreads();
            // A tile in which some row does not see some key multiplies only where the weight is not zero: 0 * inf
            // of a token that is not seen must not reach the sum.
            const bool masked = first + TK > p.end || (p.seg >= a.n_groups && first + TK > p.g.ctx);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float al = row_a[rg * 4 + r];
#pragma unroll
                for (int c = 0; c < S::NC; ++c) {
                    acc[r][c].x *= al;
                    acc[r][c].y *= al;
                    acc[r][c].z *= al;
                    acc[r][c].w *= al;
                }
            }
            auto weigh = [&](auto guard) {
                for (int k4 = ks * 4; k4 < TK; k4 += 4 * S::KS) {
                    float4 pw[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) pw[r] = *reinterpret_cast<const float4 *>(ss + (rg * 4 + r) * S::SP + k4);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
#pragma unroll
                        for (int c = 0; c < S::NC; ++c) {
                            const float4 v = lds4<ES>(tv + (size_t)(k4 + u) * S::ROW + (cx + c * S::TPR) * 4 * ES);
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float e = u == 0 ? pw[r].x : u == 1 ? pw[r].y : u == 2 ? pw[r].z : pw[r].w;
                                if (!guard.value || e != 0.0f) {
                                    acc[r][c].x = fmaf(e, v.x, acc[r][c].x);
                                    acc[r][c].y = fmaf(e, v.y, acc[r][c].y);
                                    acc[r][c].z = fmaf(e, v.z, acc[r][c].z);
                                    acc[r][c].w = fmaf(e, v.w, acc[r][c].w);
                                }
                            }
                        }
                    }
                }
            };
            if (masked) weigh(std::true_type{});
            else weigh(std::false_type{});
            __syncthreads();
        }
        // join the threads that split the keys
        if constexpr (S::KS > 1) {
            float *red = reinterpret_cast<float *>(smem + S::OFF_K);   // [KS - 1][TM][DP]: the key buffers are free
            static_assert((size_t)(S::KS - 1) * TM * DP * 4 <= S::OFF_S - S::OFF_K, "fits the key and value buffers");
            if (ks > 0) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<float4 *>(red + ((size_t)(ks - 1) * TM + rg * 4 + r) * DP + cx * 4) = acc[r][0];
            }
            __syncthreads();
            if (ks == 0) {
#pragma unroll
                for (int j = 0; j < S::KS - 1; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float4 o = *reinterpret_cast<const float4 *>(red + ((size_t)j * TM + rg * 4 + r) * DP + cx * 4);
                        acc[r][0].x += o.x;
                        acc[r][0].y += o.y;
                        acc[r][0].z += o.z;
                        acc[r][0].w += o.w;
                    }
            }
        }
        const bool whole = p.k0 == 0 && p.k1 == p.kt && p.seg >= a.n_groups && seg_alone(p.g);
        const size_t slot = unit_slot(a, a.geo, p.g, p.seg < a.n_groups, h, p.t) + (size_t)blockIdx.x * TM;
        if (ks == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = rg * 4 + r;
                if (m >= p.vr) continue;
                const float l = row_l[m], inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
                const int i = (m0 + m) / a.G, g = m0 + m - i * a.G;
                char *dst = a.out + (int64_t)(p.g.r0 + i) * a.o_row + (int64_t)(h * a.G + g) * a.o_head;
#pragma unroll
                for (int c = 0; c < S::NC; ++c) {
                    const int col = cx + c * S::TPR;
                    if (col >= D4) continue;
                    float4 o = acc[r][c];
                    if (!whole) {
                        *reinterpret_cast<float4 *>(a.part + (slot + m) * D + col * 4) = o;
                    } else if constexpr (ES == 4) {
                        *reinterpret_cast<float4 *>(dst + col * 16) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                    } else {
                        const float f[8] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv, 0.f, 0.f, 0.f, 0.f};
                        const uint4 wv = pack16<2>(f);
                        *reinterpret_cast<uint2 *>(dst + col * 8) = make_uint2(wv.x, wv.y);
                    }
                }
            }
        }
        if (tid < p.vr) {
            if (!whole) {
                a.part_ml[slot + tid] = make_float2(row_m[tid], row_l[tid]);
            } else if (a.lse) {
                const int i = (m0 + tid) / a.G, g = m0 + tid - i * a.G;
                const float l = row_l[tid];
                a.lse[(size_t)(p.g.r0 + i) * a.q_heads + h * a.G + g] = l == 0.0f ? -INFINITY : (row_m[tid] + log2f(l)) / kLog2e;
            }
        }
        __syncthreads();
    }
}

constexpr size_t kNoSlot = ~(size_t)0;   // a block whose range holds no tile of the unit

// Adds the pieces of one row, a warp: out = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p over n blocks, in order; slot_of(p) is
// the p-th one's slot.  Lanes take the pieces' maxima and sums, then the row's elements.
template <int ES, class F>
__device__ __forceinline__ void join_row(const AttendArgs &a, int row, int qh, int n, int lane, F slot_of) {
    const int D = a.c.head_dim, D4 = D / 4;
    float m = -INFINITY, l = 0.0f;
    float4 o[2] = {};
    for (int base = 0; base < n; base += 32) {
        const int p = base + lane;
        const size_t slot = p < n ? slot_of(p) : kNoSlot;
        const float2 ml = slot != kNoSlot ? a.part_ml[slot] : make_float2(-INFINITY, 0.0f);
        float top = ml.y == 0.0f ? -INFINITY : ml.x;   // a piece whose tokens the row did not see adds nothing
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        top = fmaxf(top, m);
        const float ref = top == -INFINITY ? 0.0f : top;
        const float w = ml.y == 0.0f ? 0.0f : exp2f(ml.x - ref), before = exp2f(m - ref);
        float sum = w * ml.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        l = l * before + sum;
        m = top;
#pragma unroll
        for (int j = 0; j < 2; ++j) o[j] = make_float4(o[j].x * before, o[j].y * before, o[j].z * before, o[j].w * before);
        const int many = min(32, n - base);
#pragma unroll 4
        for (int q = 0; q < many; ++q) {
            const float f = __shfl_sync(0xFFFFFFFFu, w, q);
            const size_t at = __shfl_sync(0xFFFFFFFFu, slot, q) * D;
            if (f != 0.0f) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = lane + 32 * j;
                    if (col < D4) {
                        const float4 x = *reinterpret_cast<const float4 *>(a.part + at + col * 4);
                        o[j].x = fmaf(x.x, f, o[j].x);
                        o[j].y = fmaf(x.y, f, o[j].y);
                        o[j].z = fmaf(x.z, f, o[j].z);
                        o[j].w = fmaf(x.w, f, o[j].w);
                    }
                }
            }
        }
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    char *dst = a.out + (int64_t)row * a.o_row + (int64_t)qh * a.o_head;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int col = lane + 32 * j;
        if (col >= D4) continue;
        const float4 x = make_float4(o[j].x * inv, o[j].y * inv, o[j].z * inv, o[j].w * inv);
        if constexpr (ES == 4) {
            *reinterpret_cast<float4 *>(dst + col * 16) = x;
        } else {
            const float f[8] = {x.x, x.y, x.z, x.w, 0.f, 0.f, 0.f, 0.f};
            const uint4 wv = pack16<2>(f);
            *reinterpret_cast<uint2 *>(dst + col * 8) = make_uint2(wv.x, wv.y);
        }
    }
    if (a.lse && lane == 0) a.lse[(size_t)row * a.q_heads + qh] = l == 0.0f ? -INFINITY : (m + log2f(l)) / kLog2e;
}

// Without prefixes: the units that several blocks share, one block of the grid eight rows of a tail.
template <int ES>
__global__ void __launch_bounds__(256) k_attend_join_tails(const AttendArgs a) {
    pdl_wait();
    const AttendTail t = a.tails[blockIdx.x];
    const int lane = threadIdx.x & 31, m = blockIdx.y * 8 + (threadIdx.x >> 5);
    if (m >= t.vr || t.tiles == 0) return;
    const int i = (t.m0 + m) / a.G, g = t.m0 + m - i * a.G;
    const Ranges r = ranges_of(t.total, a.geo);
    const int c0 = block_of_place(r, t.at);
    join_row<ES>(a, t.r0 + i, t.h * a.G + g, (int)blockIdx.x - c0 + 1, lane, [&](int p) {
        return block_has(r, c0 + p, t.at, t.cost, t.tiles) ? (size_t)t.slot + m + (size_t)(c0 + p) * a.geo.TM : kNoSlot;
    });
}

// With prefixes: every row adds those of its group's prefix, then its own.  A block takes kJoinRows packed rows of one
// (sequence, key head); its segments are looked up once, its rows' pieces by a lane each.
constexpr int kJoinRows = 8;

template <int ES>
__global__ void __launch_bounds__(256) k_attend_join(const AttendArgs a, const AttendGeo prefix, const AttendGeo own) {
    __shared__ JoinSeg sj[2];
    pdl_wait();
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int h = blockIdx.x % a.c.kv_heads, unit = blockIdx.x / a.c.kv_heads;
    const bool ragged = a.bt.row_start != nullptr;   // then a block takes the heads of one row
    const int b = ragged ? row_sequence(a.bt, unit) : unit;
    if (threadIdx.x == 0) sj[1] = join_seg(a, own, a.n_groups + b, h);
    if (threadIdx.x == 32) sj[0] = join_seg(a, prefix, group_of(a, b), h);
    __syncthreads();
    const JoinSeg &jo = sj[1], &jp = sj[0];
    const int start = ragged ? (unit - jo.g.r0) * a.G : blockIdx.y * kJoinRows;
    const int stop = start < 0 ? start : ragged ? min(jo.g.packed, start + a.G) : jo.g.packed;
    const int stride = ragged ? 8 : (int)gridDim.y * kJoinRows;   // rows go kJoinRows (ragged: a.G) at a time, a warp each
    for (int mm = start + wp; mm < stop; mm += stride) {
        const int i = mm / a.G, row = jo.g.r0 + i, qh = h * a.G + mm - i * a.G;
        const int to = mm / own.TM;
        const JoinUnit uo = join_unit(a, own, jo, to);
        if (uo.c0 == uo.c1 && seg_alone(jo.g)) continue;   // written by its piece
        JoinUnit up{0, 1, 0, 0, -1};
        size_t sp = 0;
        if (row >= jp.g.r0 && row < jp.g.r0 + jp.g.n) {
            const int mp = (row - jp.g.r0) * a.G + mm - i * a.G, t = mp / prefix.TM;
            up = join_unit(a, prefix, jp, t);
            sp = unit_slot(a, prefix, jp.g, true, h, t) + (mp - t * prefix.TM);
        }
        const size_t so = unit_slot(a, own, jo.g, false, h, to) + (mm - to * own.TM);
        const int np = up.c1 - up.c0 + 1;
        join_row<ES>(a, row, qh, np + (uo.c1 - uo.c0 + 1), lane, [&](int p) {
            const bool pre = p < np;
            const int c = pre ? up.c0 + p : uo.c0 + p - np;
            if (!(pre ? block_has(jp.r, c, up.at, up.cost, up.tiles) : block_has(jo.r, c, uo.at, uo.cost, uo.tiles))) return kNoSlot;
            return pre ? sp + (size_t)c * prefix.TM : so + (size_t)c * own.TM;
        });
    }
}

cudaError_t launch_attend_join(const AttendArgs &a, const AttendGeo &prefix, const AttendGeo &own, int es, cudaStream_t stream) {
    if (a.n_groups == 0) {
        const dim3 grid((unsigned)own.blocks, (unsigned)((own.TM + 7) / 8));
        return es == 4 ? launch_pdl(k_attend_join_tails<4>, grid, dim3(256), 0, stream, a)
                       : launch_pdl(k_attend_join_tails<2>, grid, dim3(256), 0, stream, a);
    }
    const dim3 grid = a.bt.row_start ? dim3((unsigned)(a.bt.rows * a.c.kv_heads))
                                     : dim3((unsigned)(a.bt.B * a.c.kv_heads), (unsigned)min(65535LL, ((long long)a.bt.n * a.G + kJoinRows - 1) / kJoinRows));
    return es == 4 ? launch_pdl(k_attend_join<4>, grid, dim3(256), 0, stream, a, prefix, own)
                   : launch_pdl(k_attend_join<2>, grid, dim3(256), 0, stream, a, prefix, own);
}

template <int ES, int DP, int TM>
static cudaError_t run_f32(AttendArgs &a, cudaStream_t stream) {
    using S = F32Shape<ES, DP, TM>;
    if (prepare_kernel((const void *)k_attend_f32<ES, DP, TM>, kAttThreads, S::BYTES) < 1) return cudaErrorInvalidConfiguration;
    constexpr AttendTiles tiles = tiles_f32(TM, DP);
    static_assert(tiles.TK == S::TK, "the cutting's key tiles are the kernel's");
    a.geo.set(tiles);
    k_attend_f32<ES, DP, TM><<<a.geo.blocks, kAttThreads, S::BYTES, stream>>>(a);
    return cudaGetLastError();
}

// `small`: tiles of kSmallRows rows.
cudaError_t launch_attend_f32(AttendArgs &a, int es, bool small, cudaStream_t stream) {
    const int D = a.c.head_dim;
#define SV_ATT(ES, DP) (small ? run_f32<ES, DP, kSmallRows>(a, stream) : run_f32<ES, DP, 64>(a, stream))
    if (es == 4) return D <= 64 ? SV_ATT(4, 64) : D <= 128 ? SV_ATT(4, 128) : SV_ATT(4, 256);
    return SV_ATT(2, 256);   // narrower bf16 heads go to the tensor cores
#undef SV_ATT
}

// Workspace of a call: segment offsets, then the slots of the widest tiles (256 rows) on the most blocks, once for the prefixes and
// once for the own tokens.
constexpr int kAttBlocks = 160;   // most persistent blocks, one an SM (a GB300 has 152); few32 has two
constexpr int kAttMaxTile = 256;

struct AttendPlan {
    size_t off_seg = 0, off_tails = 0, off_ml = 0, off_part = 0, bytes = 0;
};

static AttendPlan plan_attend(int64_t rows, int q_heads, int head_dim, int B, int n_groups) {
    AttendPlan p;
    Carver cv;
    const size_t slots = attend_slots(rows, q_heads, n_groups > 0, true, kAttMaxTile, kAttBlocks) +
                         (n_groups > 0 ? (size_t)kFewRows * kAttBlocks : 0);
    p.off_seg = cv.take<long long>((size_t)n_groups + B + 2);
    p.off_tails = cv.take<AttendTail>(2 * kAttBlocks);
    p.off_ml = cv.take<float2>(slots);
    p.off_part = cv.take<float>(slots * head_dim);
    p.bytes = cv.off + 256;
    return p;
}

// sv_selftest_attend_stall's setting of this host thread.
static thread_local long long t_stall_limit = 0;

}  // namespace sv

using namespace sv;

extern "C" void sv_selftest_attend_stall(int64_t limit_cycles) { t_stall_limit = limit_cycles; }

extern "C" size_t sv_kv_attend_workspace_size(int64_t rows, int q_heads, int head_dim, int B, int n_groups) {
    if (rows < 0 || q_heads < 1 || head_dim < 1 || head_dim > SV_KV_MAX_HEAD_DIM || B < 1 || n_groups < 0) return 0;
    return plan_attend(rows, q_heads, head_dim, B, n_groups).bytes;
}

extern "C" sv_status sv_kv_attend(const sv_kv_cache *cache, const sv_kv_batch *batch, const void *q,
                                  int64_t q_row_stride, int64_t q_head_stride, int q_heads, float scale,
                                  const int32_t *group_start, const int32_t *prefix_len, int n_groups, void *out,
                                  int64_t out_row_stride, int64_t out_head_stride, float *lse, sv_stats *stats,
                                  void *workspace, size_t workspace_bytes, sv_stream_t stream) {
    if (!kv_args_ok(cache, batch, true) || q_heads < 1 || q_heads % cache->kv_heads != 0 || !isfinite(scale))
        return SV_ERR_INVALID_ARG;
    if (n_groups < 0 || n_groups > batch->B || (n_groups > 0 && (group_start == nullptr || prefix_len == nullptr)))
        return SV_ERR_INVALID_ARG;
    const int es = elem_size((sv_dtype)cache->dtype);
    if (batch->rows > 0 && (q == nullptr || out == nullptr)) return SV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !strides16(es, q_row_stride, q_head_stride) ||
        !strides16(es, out_row_stride, out_head_stride) || (int64_t)batch->rows * q_heads > (1 << 30) ||
        (int64_t)batch->B * cache->kv_heads > INT32_MAX)
        return SV_ERR_INVALID_ARG;
    // Rows that meet the same tokens, and the tiles they are cut into (few rows make one row tile, which always fits).
    const bool fma = es == 4 || cache->head_dim > 128;
    const int64_t G = q_heads / cache->kv_heads, packed = batch->n * G;
    const bool few = packed <= (fma ? kSmallRows : kFewRows);
    const AttendTiles large = fma ? tiles_f32(64, cache->head_dim > 128 ? 256 : 128) : kTilesTall;
    if ((!few || n_groups > 0) &&
        !tiles_fit(large, (n_groups > 0 || batch->rows < batch->n ? batch->rows : batch->n) * G, (int64_t)batch->max_pages * cache->page_size))
        return SV_ERR_INVALID_ARG;
    const AttendPlan pl = plan_attend(batch->rows, q_heads, cache->head_dim, batch->B, n_groups);
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < pl.bytes) return SV_ERR_WORKSPACE;
    const int64_t width = (int64_t)cache->head_dim * es;
    if (overlap({q, q_row_stride * es, q_head_stride * es, batch->rows, q_heads, width},
                {out, out_row_stride * es, out_head_stride * es, batch->rows, q_heads, width}))
        return SV_ERR_INVALID_ARG;   // other blocks still read q
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on_current_device(s, cache->k, q)) return SV_ERR_INVALID_ARG;
    DeviceInfo di;
    if (!device_info(di)) return SV_ERR_CUDA;
    if (stats && cudaMemsetAsync(stats, 0, sizeof(sv_stats), s) != cudaSuccess) return SV_ERR_CUDA;
    if (batch->rows == 0) return SV_OK;
    char *w = static_cast<char *>(workspace);
    AttendArgs a{};
    a.c = kv_cache_of(*cache);
    a.bt = kv_batch_of(*batch);
    a.q = static_cast<const char *>(q);
    a.out = static_cast<char *>(out);
    a.q_row = q_row_stride * es;
    a.q_head = q_head_stride * es;
    a.o_row = out_row_stride * es;
    a.o_head = out_head_stride * es;
    a.q_heads = q_heads;
    a.G = q_heads / cache->kv_heads;
    a.scale_log2 = (float)((double)scale * 1.44269504088896340736);
    a.group_start = group_start;
    a.prefix_len = prefix_len;
    a.n_groups = n_groups;
    a.lse = lse;
    a.stats = stats;
    a.wait_limit = t_stall_limit > 0 ? t_stall_limit : kWaitLimitCycles;
    a.stuck_stage = t_stall_limit > 0 ? 2 : -1;
    a.tails = reinterpret_cast<AttendTail *>(w + pl.off_tails);
    a.part_ml = reinterpret_cast<float2 *>(w + pl.off_ml);
    a.part = reinterpret_cast<float *>(w + pl.off_part);
    long long *seg = reinterpret_cast<long long *>(w + pl.off_seg);
    const int blocks = di.sms < kAttBlocks ? di.sms : kAttBlocks;
    const AttendGeo all{0, n_groups + batch->B, 0, 0, blocks, 1, 1, 0, seg, 0};
    AttendGeo prefix = all, own = all;
    cudaError_t e = cudaSuccess;
    // bf16 heads up to 128 wide go to the tensor cores; wider ones have float32 arithmetic only (two outputs of 256 columns would fill
    // the tall kernel's tensor memory, and no other form is built).  Where a sequence's own
    // tokens meet few packed rows they have a kernel of their own: up to 32 rows on the tensor cores, with the tokens along the
    // tile's rows (512 x 6 rows over 1-2k tokens: 525 us, against 1,040 in the tall kernel); up to 8 in float32 by warps (64 single
    // tokens of 4 rows: 112 us, against 360 in tiles); up to 16 otherwise in tiles of 16 rows.  Beside prefixes too, in a second
    // launch: 64 x 16 float32 rows over 1.9-3.5k own tokens take 676 us, in the prefixes' tiles of 64 rows 2,230.  On the tensor cores
    // 64 x 6 rows behind 32k tokens would take 266 us in one launch instead of 291, but twice as long where own tokens outweigh the
    // prefix, and the lengths are on the device.
    a.geo = all;
    if (!few || n_groups > 0) {
        if (few) a.geo.s1 = n_groups;
        e = fma ? launch_attend_f32(a, es, false, s) : launch_attend_tall(a, s);
        prefix = own = a.geo;
    }
    if (few && e == cudaSuccess) {
        a.geo = all;
        if (n_groups > 0) {
            a.geo.s0 = n_groups;
            a.geo.seg_off = seg + n_groups + 1;
            a.geo.slot0 = attend_slots(batch->rows, q_heads, true, false, prefix.TM, blocks);
        }
        e = !fma ? launch_attend_few(a, s)
            : es == 4 && cache->head_dim <= 128 && packed <= kFewRows32 ? launch_attend_few32(a, s)
                                                                         : launch_attend_f32(a, es, true, s);
        own = a.geo;
    }
    if (e == cudaSuccess) e = launch_attend_join(a, prefix, own, es, s);
    return cuda_status(e);
}
