// sv_kv8.cu — the append to a paged cache held in 8 bits, and the commit of an accepted path in it.
#include <math.h>

#include "sv_code8.cuh"

namespace sv {

namespace {

constexpr int kHeadGroup = 8;    // key heads of a block, a warp each
constexpr int kAppendThreads = 32 * kHeadGroup;
constexpr int kChunk = 8;        // tokens whose angles are held at a time

struct Append8Args {
    KvCache c;
    uint8_t *k_scale, *v_scale;
    int64_t scale_page, scale_head;
    KvBatch bt;
    const char *q, *k, *v;
    char *q_out;
    int64_t q_row, q_head, qo_row, qo_head, k_row, k_head, v_row, v_head;   // bytes
    const float *inv_freq;
    RotShape sh;     // heads = query heads
    float magnitude;
    sv_stats *stats;
};

// The elements that item i of a head covers (rot_item's items), rotated: E of them from e0 in x, and in the half style the E that
// they pair up with from e1 in y (e1 < 0: none).
template <int ES, bool VEC>
__device__ __forceinline__ void rot_values(const RotShape &s, const char *src, int i, const float2 *cs, float *x, float *y, int &e0, int &e1) {
    constexpr int E = VEC ? 16 / ES : 1;
    auto load = [&](int e, float *to) {
        if constexpr (VEC) {
            float t[E];
            unpack<ES>(*reinterpret_cast<const uint4 *>(src + (size_t)e * ES), t);
#pragma unroll
            for (int j = 0; j < E; ++j) to[j] = t[j];
        } else {
            to[0] = load_elem<ES>(src, e);
        }
    };
    const bool inter = s.style == SV_ROPE_INTERLEAVED;
    const int turned = s.half == 0 ? 0 : VEC && inter ? 2 * s.half / E : s.half / E;
    e1 = -1;
    if (i >= turned) {
        e0 = 2 * s.half + (i - turned) * E;
        load(e0, x);
    } else if (VEC && inter) {
        e0 = i * E;
        load(e0, x);
#pragma unroll
        for (int j = 0; j + 1 < E; j += 2) {
            const float2 c = cs[e0 / 2 + j / 2];
            const float u = x[j], w = x[j + 1];
            x[j] = __fmaf_rn(u, c.x, -__fmul_rn(w, c.y));
            x[j + 1] = __fmaf_rn(u, c.y, __fmul_rn(w, c.x));
        }
    } else {
        e0 = inter ? 2 * i : i * E;
        e1 = inter ? 2 * i + 1 : e0 + s.half;
        load(e0, x);
        load(e1, y);
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const float2 c = cs[i * E + j];
            const float u = x[j], w = y[j];
            x[j] = __fmaf_rn(u, c.x, -__fmul_rn(w, c.y));
            y[j] = __fmaf_rn(u, c.y, __fmul_rn(w, c.x));
        }
    }
}

// x / scale, as one code a byte (inv is 1 / scale, a power of two: the product is exact where it matters).  Infinities become NaN.
template <int E>
__device__ __forceinline__ void store_codes(char *dst, const float *x, float inv) {
    float y[E];
#pragma unroll
    for (int j = 0; j < E; ++j) y[j] = fabsf(x[j]) == INFINITY ? NAN : x[j] * inv;
    if constexpr (E == 1) {
        *reinterpret_cast<uint8_t *>(dst) = (uint8_t)to_codes2(y[0], 0.0f);
    } else if constexpr (E == 4) {
        *reinterpret_cast<uint32_t *>(dst) = to_codes2(y[0], y[1]) | to_codes2(y[2], y[3]) << 16;
    } else {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(to_codes2(y[0], y[1]) | to_codes2(y[2], y[3]) << 16,
                                                     to_codes2(y[4], y[5]) | to_codes2(y[6], y[7]) << 16);
    }
}

template <int E>
__device__ __forceinline__ float most_finite(const float *x) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const float a = fabsf(x[j]);
        m = fmaxf(m, a < INFINITY ? a : 0.0f);
    }
    return m;
}

__device__ __forceinline__ void prefetch_l1(const char *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// The first row that a page gets takes that page's keys and values, a warp to each of eight key heads: the largest element, the page's
// scale from it, then the codes.  Keys are rotated twice, once for each, from the first-level cache the second time.  Every row
// takes its queries, an equal part a group of heads.
//
// Bound by latency and instruction issue, not by bytes: a scale needs the page's whole part of the block before its first code, and an
// element is read, turned, looked at, turned again and rounded.  512 sequences x 6 rows, 32 + 8 + 8 heads of 128, bf16: 36 us, 10.4 us at the
// memory's rate.  What it reads is asked for before the addresses that hang on the context length are known (42 us without); a
// block for keys and one for values instead of one for both: 37.6 us; a block's maxima joined in shared memory: 37 us; blocks of 64 threads: 43 us.
template <int ES, bool VEC>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append8(const Append8Args a) {
    constexpr int E = VEC ? 16 / ES : 1, EV = 16 / ES;
    __shared__ float2 cs[kChunk][SV_KV_MAX_HEAD_DIM / 2];
    __shared__ int32_t par[SV_MAX_TREE];
    __shared__ int s_depth[kChunk];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x, group = blockIdx.y, groups = gridDim.y, h = group * kHeadGroup + warp;
    const int q0 = (int)((int64_t)a.sh.heads * group / groups), q1 = (int)((int64_t)a.sh.heads * (group + 1) / groups);
    const int lines = (a.c.head_dim * ES + 127) / 128;   // of a head
    if (a.q != nullptr)
        for (int t = tid; t < (q1 - q0) * lines; t += kAppendThreads) {
            const int h = t / lines;
            prefetch_l1(a.q + (int64_t)row * a.q_row + (q0 + h) * a.q_head + (t - h * lines) * 128);
        }
    const int b = row_sequence(a.bt, row);
    const SeqRows sr = seq_rows(a.bt, b);
    const int i = row - sr.r0, ctx = a.bt.context_len[b];
    const int64_t cap = (int64_t)a.bt.max_pages * a.c.page_size;
    if (!sr.ok || ctx < 0 || ctx + (int64_t)sr.n > cap) {
        if (tid == 0) report_error(a.stats, SV_ERR_INVALID_ARG, b);
        return;
    }
    if (i < 0 || i >= sr.n) return;   // a row of no sequence
    const int psize = a.c.page_size, slot0 = ctx + i, pn = slot0 / psize, place0 = slot0 - pn * psize;
    const bool leads = i == 0 || place0 == 0;
    if (!leads && a.q == nullptr) return;
    const int T = leads ? min(sr.n - i, psize - place0) : 1;   // rows of the page
    if (leads && h < a.c.kv_heads)
        for (int t = lane; t < 2 * lines * min(T, 16); t += 32) {
            const int r = t / (2 * lines), l = t - r * 2 * lines;
            const char *head = l < lines ? a.v + (int64_t)(row + r) * a.v_row + h * a.v_head : a.k + (int64_t)(row + r) * a.k_row + h * a.k_head;
            prefetch_l1(head + (l < lines ? l : l - lines) * 128);
        }
    const int page = leads ? a.bt.page_table[b * a.bt.table_pitch + pn] : -1;
    if (leads && (page < 0 || page >= a.c.n_pages) && tid == 0) report_error(a.stats, SV_ERR_INVALID_ARG, b);
    if (a.bt.parents != nullptr) {
        for (int j = tid; j < i + T - 1; j += kAppendThreads) par[j] = a.bt.parents[(int64_t)b * (a.bt.n - 1) + j];
        __syncthreads();
    }

    auto angles = [&](int t0, int n) {   // rows i + t0 .. i + t0 + n - 1
        if (tid < n) {
            const int r = i + t0 + tid;
            int depth = r;
            if (a.bt.parents != nullptr) {
                depth = 0;
                for (int j = r; j > 0; ++depth) {
                    const int p = par[j - 1];
                    if (p < 0 || p >= j) {
                        report_error(a.stats, SV_ERR_INVALID_ARG, b);
                        break;
                    }
                    j = p;
                }
            }
            s_depth[tid] = depth;
        }
        __syncthreads();
        for (int t = warp; t < n; t += kHeadGroup) {
            const int at = ctx + s_depth[t];
            for (int f = lane; f < a.sh.half; f += 32) {
                const float2 c = rope_cos_sin(at, a.inv_freq[f]);
                cs[t][f] = make_float2(c.x * a.magnitude, c.y * a.magnitude);
            }
        }
        __syncthreads();
    };

    const int per = rot_items<ES, VEC>(a.sh);   // items of a rotated head
    angles(0, min(T, kChunk));
    if (a.q != nullptr) {
        for (int t = tid; t < per * (q1 - q0); t += kAppendThreads) {
            const int h = q0 + t / per;
            rot_item<ES, VEC>(a.sh, a.q + (int64_t)row * a.q_row + h * a.q_head, a.q_out + (int64_t)row * a.qo_row + h * a.qo_head, t % per,
                              cs[0]);
        }
    }
    if (page < 0 || page >= a.c.n_pages) return;

    // use(token, item) for the `of` items a token of n tokens, each by one lane.
    auto each = [&](int n, int of, auto &&use) {
        const int dt = 32 / of, di = 32 - dt * of;
        int t = lane / of, w = lane - t * of;
#pragma unroll 2
        while (t < n) {
            use(t, w);
            t += dt;
            w += di;
            if (w >= of) {
                w -= of;
                ++t;
            }
        }
    };
    const bool fresh = place0 == 0, mine = h < a.c.kv_heads;   // no cached token in the page; a warp with a head
    auto scale_at = [&](uint8_t *scales) { return scales + page * a.scale_page + h * a.scale_head; };
    // The page's scale from the largest element that a lane has seen; `shift`: by how much the cached tokens' codes go down.
    auto settle = [&](uint8_t *at, float most, int old, int &shift) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        const int byte = max(scale_for(most), old);
        shift = fresh ? 0 : byte - old;
        __syncwarp();   // every lane has read the scale
        if (lane == 0 && (fresh || shift > 0)) *at = (uint8_t)byte;
        return byte;
    };
    auto inverse = [](int byte) { return scale_of(byte == 255 ? 255 : 254 - byte); };
    auto cached = [&](char *codes, int shift) {   // the page's cached tokens, where the scale has grown
        if (shift <= 0) return;
        each(place0, a.c.head_dim / 16, [&](int t, int w) {
            uint4 *at = reinterpret_cast<uint4 *>(codes + t * a.c.slot_b + w * 16);
            *at = rescaled16(*at, shift);
        });
    };
    const int64_t to = page * a.c.page_b + h * a.c.head_b;
    if (mine) {
        const char *src = a.v + (int64_t)row * a.v_row + h * a.v_head;
        uint8_t *at = scale_at(a.v_scale);
        const int old = fresh ? 0 : *at;
        float most = 0.0f;
        auto load = [&](int t, int w, float (&x)[EV]) { unpack<ES>(*reinterpret_cast<const uint4 *>(src + t * a.v_row + w * 16), x); };
        each(T, a.c.head_dim / EV, [&](int t, int w) {
            float x[EV];
            load(t, w, x);
            most = fmaxf(most, most_finite<EV>(x));
        });
        int shift;
        const float inv = inverse(settle(at, most, old, shift));
        each(T, a.c.head_dim / EV, [&](int t, int w) {
            float x[EV];
            load(t, w, x);
            store_codes<EV>(a.c.v + to + (place0 + t) * a.c.slot_b + w * EV, x, inv);
        });
        cached(a.c.v + to, shift);
    }
    {
        const char *src = a.k + (int64_t)row * a.k_row + h * a.k_head;
        uint8_t *at = scale_at(a.k_scale);
        const int old = mine && !fresh ? *at : 0;
        float most = 0.0f, x[E], y[E];
        int e0, e1, shift = 0;
        auto chunks = [&](bool again, auto &&use) {   // use(token): the element of x, y at e0, e1
            for (int t0 = 0; t0 < T; t0 += kChunk) {
                const int n = min(T - t0, kChunk);
                if (t0 > 0 || (again && T > kChunk)) {
                    __syncthreads();
                    angles(t0, n);
                }
                if (mine)
                    each(n, per, [&](int t, int w) {
                        rot_values<ES, VEC>(a.sh, src + (t0 + t) * a.k_row, w, cs[t], x, y, e0, e1);
                        use(t0 + t);
                    });
            }
        };
        chunks(false, [&](int) {
            most = fmaxf(most, most_finite<E>(x));
            if (e1 >= 0) most = fmaxf(most, most_finite<E>(y));
        });
        float inv = 0.0f;
        if (mine) inv = inverse(settle(at, most, old, shift));
        chunks(true, [&](int t) {
            char *codes = a.c.k + to + (place0 + t) * a.c.slot_b;
            store_codes<E>(codes + e0, x, inv);
            if (e1 >= 0) store_codes<E>(codes + e1, y, inv);
        });
        cached(a.c.k + to, shift);
    }
}

struct Commit8Args {
    KvCache c;
    uint8_t *k_scale, *v_scale;
    int64_t scale_page, scale_head;
    KvBatch bt;
    int64_t layer_b, scale_layer_b;
    const int32_t *accept_len, *path;
    int32_t *context_out;
    sv_stats *stats;
};

// One block a (layer, sequence), as in k_kv_commit; thread t holds one 16-byte column of a head's codes.  Destinations rise and no source lies before
// its destination, so pages are finished one after the other, and a page's own scale is needed by nothing that comes later.  All
// threads read the scales as they were; the new ones are written at the end.
// Bound by latency: table, scales and codes are loads that follow one another, for a few moves a block.  32 layers x 64 sequences, trees of
// 57: 12.1 us in a graph, 4.4 us at the memory's rate (k_kv_commit: 12 us for twice the bytes).
__global__ void __launch_bounds__(256) k_kv_commit8(const Commit8Args a) {
    __shared__ int64_t src[SV_MAX_TREE], dst[SV_MAX_TREE];
    __shared__ int32_t src_page[SV_MAX_TREE], dst_page[SV_MAX_TREE];
    const int b = blockIdx.x % a.bt.B, N = a.bt.n - 1;
    const int64_t layer = blockIdx.x / a.bt.B;
    const int acc = a.accept_len[b], ctx = a.bt.context_len[b], psize = a.c.page_size;
    const int32_t *path = a.path + (int64_t)b * N;
    const SeqRows sr = seq_rows(a.bt, b);
    const int64_t cap = (int64_t)a.bt.max_pages * psize;
    bool bad = !sr.ok || acc < 0 || acc > max(sr.n - 1, 0) || ctx < 0 || ctx + (int64_t)min(sr.n, 1) > cap;
    if (!bad) {
        const int32_t *table = a.bt.page_table + b * a.bt.table_pitch;
        for (int j = threadIdx.x; j < acc; j += 256) {
            const int p = path[j];
            if (p >= sr.n || ctx + (int64_t)p >= cap || p <= (j ? path[j - 1] : 0) || p <= j) {
                bad = true;
            } else {
                src[j] = slot_offset(a.c, table, ctx + p);
                dst[j] = slot_offset(a.c, table, ctx + 1 + j);
                if (src[j] < 0 || dst[j] < 0) {
                    bad = true;
                } else {
                    src_page[j] = table[(ctx + p) / psize];
                    dst_page[j] = table[(ctx + 1 + j) / psize];
                }
            }
        }
    }
    bad = __syncthreads_or(bad);
    if (layer == 0 && threadIdx.x == 0) {
        if (bad) report_error(a.stats, SV_ERR_INVALID_ARG, b);
        if (a.context_out) a.context_out[b] = bad || sr.n == 0 ? ctx : ctx + 1 + acc;
    }
    if (bad || acc == 0) return;
    const int vec = a.c.head_dim / 16, cols = vec * a.c.kv_heads;
    const int first_place = (ctx + 1) % psize;   // of the first move's destination: slots before it hold tokens
    auto scales = [&](int which, int h) { return (which ? a.v_scale : a.k_scale) + layer * a.scale_layer_b + h * a.scale_head; };
    // Moves [j, returned) share a destination page; `byte` is the scale it gets.
    auto page_moves = [&](const uint8_t *scale, int j, int &byte) {
        const int in_page = psize - (ctx + 1 + j) % psize, end = min(acc, j + in_page);
        byte = scale[dst_page[j] * a.scale_page];
        for (int m = j; m < end; ++m) byte = max(byte, (int)scale[src_page[m] * a.scale_page]);
        return end;
    };
    for (int t = threadIdx.x; t < 2 * cols; t += 256) {
        const int which = t >= cols, u = t - which * cols, h = u / vec;
        const uint8_t *scale = scales(which, h);
        char *base = (which ? a.c.v : a.c.k) + layer * a.layer_b + h * a.c.head_b + (u - h * vec) * 16;
        for (int j = 0; j < acc;) {
            int byte;
            const int end = page_moves(scale, j, byte), grown = byte - scale[dst_page[j] * a.scale_page];
            if (j == 0 && grown > 0) {
                char *at = base + dst_page[0] * a.c.page_b;
                for (int s = 0; s < first_place; ++s, at += a.c.slot_b)
                    *reinterpret_cast<uint4 *>(at) = rescaled16(*reinterpret_cast<const uint4 *>(at), grown);
            }
            for (; j < end; ++j) {
                const int shift = byte - scale[src_page[j] * a.scale_page];
                if (src[j] != dst[j] || shift > 0)
                    *reinterpret_cast<uint4 *>(base + dst[j]) = rescaled16(*reinterpret_cast<const uint4 *>(base + src[j]), shift);
            }
        }
    }
    __syncthreads();
    for (int t = threadIdx.x; t < 2 * a.c.kv_heads; t += 256) {
        const int which = t >= a.c.kv_heads, h = t - which * a.c.kv_heads;
        uint8_t *scale = scales(which, h);
        for (int j = 0; j < acc;) {
            int byte;
            const int at = dst_page[j];
            j = page_moves(scale, j, byte);
            if (scale[at * a.scale_page] != byte) scale[at * a.scale_page] = (uint8_t)byte;
        }
    }
}

}  // namespace

}  // namespace sv

using namespace sv;

extern "C" sv_status sv_kv_append8(const sv_kv_cache8 *cache, const sv_kv_batch *batch, sv_dtype dtype, const void *q,
                                   int64_t q_row_stride, int64_t q_head_stride, void *q_out, int64_t q_out_row_stride,
                                   int64_t q_out_head_stride, int q_heads, const void *k, int64_t k_row_stride,
                                   int64_t k_head_stride, const void *v, int64_t v_row_stride, int64_t v_head_stride,
                                   const float *inv_freq, int rotary_dim, int style, float magnitude, sv_stats *stats,
                                   sv_stream_t stream) {
    if (!kv_args_ok(cache, batch, dtype, true) || !rope_args_ok(inv_freq, rotary_dim, style, cache->head_dim)) return SV_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (q != nullptr && q_heads < 1)) return SV_ERR_INVALID_ARG;
    const int es = elem_size(dtype);
    if (batch->rows > 0 && (k == nullptr || v == nullptr)) return SV_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !strides16(es, k_row_stride, k_head_stride) || !strides16(es, v_row_stride, v_head_stride))
        return SV_ERR_INVALID_ARG;
    if (q != nullptr && (!strides16(es, q_row_stride, q_head_stride) || !strides16(es, q_out_row_stride, q_out_head_stride)))
        return SV_ERR_INVALID_ARG;
    const int64_t width = (int64_t)cache->head_dim * es;
    if (q != nullptr && turns_onto({q, q_row_stride * es, q_head_stride * es, batch->rows, q_heads, width},
                                   {q_out, q_out_row_stride * es, q_out_head_stride * es, batch->rows, q_heads, width}))
        return SV_ERR_INVALID_ARG;
    const int groups = (cache->kv_heads + kHeadGroup - 1) / kHeadGroup;
    if (groups > 65535) return SV_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on_current_device(s, cache->k, k)) return SV_ERR_INVALID_ARG;
    if (stats && cudaMemsetAsync(stats, 0, sizeof(sv_stats), s) != cudaSuccess) return SV_ERR_CUDA;
    if (batch->rows == 0) return SV_OK;
    Append8Args a{kv_cache_of(*cache), cache->k_scale, cache->v_scale, cache->scale_page_stride, cache->scale_head_stride, kv_batch_of(*batch),
                  static_cast<const char *>(q), static_cast<const char *>(k), static_cast<const char *>(v), static_cast<char *>(q_out),
                  q_row_stride * es, q_head_stride * es, q_out_row_stride * es, q_out_head_stride * es, k_row_stride * es, k_head_stride * es,
                  v_row_stride * es, v_head_stride * es, inv_freq, {q_heads, cache->head_dim, rotary_dim / 2, style}, magnitude, stats};
    const bool vec = rot_vec(rotary_dim / 2, style, es);
    const dim3 grid((unsigned)batch->rows, (unsigned)groups);
    if (es == 4)
        vec ? k_kv_append8<4, true><<<grid, kAppendThreads, 0, s>>>(a) : k_kv_append8<4, false><<<grid, kAppendThreads, 0, s>>>(a);
    else
        vec ? k_kv_append8<2, true><<<grid, kAppendThreads, 0, s>>>(a) : k_kv_append8<2, false><<<grid, kAppendThreads, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}

extern "C" sv_status sv_kv_commit8(const sv_kv_cache8 *cache, const sv_kv_batch *batch, int n_layers, int64_t layer_stride,
                                   int64_t scale_layer_stride, const int32_t *accept_len, const int32_t *path,
                                   int32_t *context_out, sv_stats *stats, sv_stream_t stream) {
    if (!kv_args_ok(cache, batch, SV_BF16, false) || n_layers < 1 || accept_len == nullptr || batch->n - 1 > SV_MAX_TREE ||
        (path == nullptr && batch->n > 1) || context_out == batch->context_len)
        return SV_ERR_INVALID_ARG;
    if (layer_stride % 16 != 0 || (int64_t)batch->B * n_layers > INT32_MAX) return SV_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on_current_device(s, cache->k, accept_len)) return SV_ERR_INVALID_ARG;
    if (stats && cudaMemsetAsync(stats, 0, sizeof(sv_stats), s) != cudaSuccess) return SV_ERR_CUDA;
    const Commit8Args a{kv_cache_of(*cache), cache->k_scale, cache->v_scale, cache->scale_page_stride, cache->scale_head_stride,
                        kv_batch_of(*batch), layer_stride, scale_layer_stride, accept_len, path, context_out, stats};
    k_kv_commit8<<<(unsigned)(batch->B * n_layers), 256, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}
