// sv_kv.cu — rotary positions, the append to the paged cache and the commit of an accepted path.
#include <math.h>

#include "sv_kv.cuh"

namespace sv {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    const char *x;
    char *out;
    int64_t x_row, x_head, o_row, o_head;   // bytes
    const int32_t *positions;
    const float *inv_freq;
    RotShape sh;
    float magnitude, sign;
};

// One block a row: its angles once, for all heads.  Memory bounds it: 8,192 rows of 32 heads of 128, bf16, take 24.9 us, 5.4 TB/s or
// 0.79 of the measured copy bandwidth.  (Loading a thread's first item before the angles cost registers and took 27.2 us.)
template <int ES, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const RopeArgs a) {
    __shared__ float2 cs[SV_KV_MAX_HEAD_DIM / 2];
    const int64_t r = blockIdx.x;
    for (int i = threadIdx.x; i < a.sh.half; i += kRopeThreads) {
        const float2 c = rope_cos_sin(a.positions[r], a.inv_freq[i]);
        cs[i] = make_float2(c.x * a.magnitude, c.y * a.magnitude * a.sign);
    }
    __syncthreads();
    const int per = rot_items<ES, VEC>(a.sh), all = per * a.sh.heads;
    for (int i = threadIdx.x; i < all; i += kRopeThreads) {
        const int h = i / per;
        rot_item<ES, VEC>(a.sh, a.x + r * a.x_row + h * a.x_head, a.out + r * a.o_row + h * a.o_head, i - h * per, cs);
    }
}

struct AppendArgs {
    KvCache c;
    KvBatch bt;
    const char *q, *k, *v;
    char *q_out;
    int64_t q_row, q_head, qo_row, qo_head, k_row, k_head, v_row, v_head;   // bytes
    const float *inv_freq;
    RotShape sh;     // heads = query heads
    float magnitude;
    sv_stats *stats;
};

// One block a row: the row's depth, its angles, then queries, keys and values as one list of items.  512 x 6 rows of 32 + 2 x 8 heads of
// 128, bf16: 16.3 us, 4.6 TB/s or 0.68 of the measured copy bandwidth; one block of 5 rows 3.1 us.
template <int ES, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) k_kv_append(const AppendArgs a) {
    __shared__ float2 cs[SV_KV_MAX_HEAD_DIM / 2];
    __shared__ int32_t par[SV_MAX_TREE];
    __shared__ int s_depth;
    const int row = blockIdx.x, b = row_sequence(a.bt, row);
    const SeqRows sr = seq_rows(a.bt, b);
    const int i = row - sr.r0, ctx = a.bt.context_len[b];
    const int64_t cap = (int64_t)a.bt.max_pages * a.c.page_size;
    if (!sr.ok || ctx < 0 || ctx + (int64_t)sr.n > cap) {
        if (threadIdx.x == 0) report_error(a.stats, SV_ERR_INVALID_ARG, b);
        return;
    }
    if (i < 0 || i >= sr.n) return;   // a row of no sequence
    const int64_t off = slot_offset(a.c, a.bt.page_table + b * a.bt.table_pitch, ctx + i);
    int depth = i;
    if (a.bt.parents != nullptr) {
        for (int j = threadIdx.x; j < i; j += kRopeThreads) par[j] = a.bt.parents[(int64_t)b * (a.bt.n - 1) + j];
        __syncthreads();
        if (threadIdx.x == 0) {
            int d = 0;
            for (int j = i; j > 0; ++d) {
                const int p = par[j - 1];
                if (p < 0 || p >= j) {
                    report_error(a.stats, SV_ERR_INVALID_ARG, b);
                    break;
                }
                j = p;
            }
            s_depth = d;
        }
        __syncthreads();
        depth = s_depth;
    }
    for (int j = threadIdx.x; j < a.sh.half; j += kRopeThreads) {
        const float2 c = rope_cos_sin(ctx + depth, a.inv_freq[j]);
        cs[j] = make_float2(c.x * a.magnitude, c.y * a.magnitude);
    }
    __syncthreads();
    if (off < 0 && threadIdx.x == 0) report_error(a.stats, SV_ERR_INVALID_ARG, b);
    const int per = rot_items<ES, VEC>(a.sh);
    const int nq = a.q ? per * a.sh.heads : 0, nk = per * a.c.kv_heads;
    const int vvec = a.c.head_dim * ES / 16;
    const int all = nq + (off < 0 ? 0 : nk + vvec * a.c.kv_heads);
    for (int t = threadIdx.x; t < all; t += kRopeThreads) {
        if (t < nq) {
            const int h = t / per;
            rot_item<ES, VEC>(a.sh, a.q + (int64_t)row * a.q_row + h * a.q_head, a.q_out + (int64_t)row * a.qo_row + h * a.qo_head, t - h * per,
                              cs);
        } else if (t < nq + nk) {
            const int u = t - nq, h = u / per;
            rot_item<ES, VEC>(a.sh, a.k + (int64_t)row * a.k_row + h * a.k_head, a.c.k + off + h * a.c.head_b, u - h * per, cs);
        } else {
            const int u = t - nq - nk, h = u / vvec, e = (u - h * vvec) * 16;
            *reinterpret_cast<uint4 *>(a.c.v + off + h * a.c.head_b + e) =
                *reinterpret_cast<const uint4 *>(a.v + (int64_t)row * a.v_row + h * a.v_head + e);
        }
    }
}

struct CommitArgs {
    KvCache c;
    KvBatch bt;
    int64_t layer_b;
    const int32_t *accept_len, *path;
    int32_t *context_out;
    sv_stats *stats;
};

// One block a (layer, sequence): 32 layers x 64 sequences of 8 heads of 128 take 9.1 us, 0.94 of the measured copy bandwidth.  Thread t holds one 16-byte column of a slot.  Slot path[j] moves to
// slot 1 + j; the path rises, so path[j'] > 1 + j for j' > j and moves in order of j never overwrite
// a slot that a later move reads.  Only slots of the sequence's own rows are touched: a short block may end where its pages do,
// and an empty one has no row 0 to keep.
__global__ void __launch_bounds__(256, 8) k_kv_commit(const CommitArgs a, int es) {
    __shared__ int64_t src[SV_MAX_TREE], dst[SV_MAX_TREE];
    const int b = blockIdx.x % a.bt.B, N = a.bt.n - 1;
    const int64_t layer = blockIdx.x / a.bt.B;
    const int acc = a.accept_len[b], ctx = a.bt.context_len[b];
    const int32_t *path = a.path + (int64_t)b * N;
    const SeqRows sr = seq_rows(a.bt, b);
    const int64_t cap = (int64_t)a.bt.max_pages * a.c.page_size;
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
                if (src[j] < 0 || dst[j] < 0) bad = true;
            }
        }
    }
    bad = __syncthreads_or(bad);
    if (layer == 0 && threadIdx.x == 0) {
        if (bad) report_error(a.stats, SV_ERR_INVALID_ARG, b);
        if (a.context_out) a.context_out[b] = bad || sr.n == 0 ? ctx : ctx + 1 + acc;
    }
    if (bad) return;
    const int vec = a.c.head_dim * es / 16, cols = vec * a.c.kv_heads;
    for (int t = threadIdx.x; t < 2 * cols; t += 256) {
        const int u = t < cols ? t : t - cols, h = u / vec;
        char *base = (t < cols ? a.c.k : a.c.v) + layer * a.layer_b + h * a.c.head_b + (u - h * vec) * 16;
        for (int j = 0; j < acc; ++j)
            if (src[j] != dst[j]) *reinterpret_cast<uint4 *>(base + dst[j]) = *reinterpret_cast<const uint4 *>(base + src[j]);
    }
}

}  // namespace sv

using namespace sv;

extern "C" sv_status sv_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double low,
                                         double high, int64_t original_len, float *inv_freq, float *magnitude) {
    if (inv_freq == nullptr || magnitude == nullptr || rotary_dim < 2 || rotary_dim % 2 != 0 ||
        rotary_dim > SV_KV_MAX_HEAD_DIM || !(base > 1.0) || !isfinite(base))
        return SV_ERR_INVALID_ARG;
    if (scaling < SV_ROPE_SCALE_NONE || scaling > SV_ROPE_SCALE_DIMS) return SV_ERR_INVALID_ARG;
    if (scaling != SV_ROPE_SCALE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return SV_ERR_INVALID_ARG;
    if (scaling == SV_ROPE_SCALE_BASE && rotary_dim < 4) return SV_ERR_INVALID_ARG;
    if (scaling >= SV_ROPE_SCALE_TURNS &&
        (!(low < high) || !isfinite(low) || !isfinite(high) || original_len < 1 ||
         (scaling == SV_ROPE_SCALE_DIMS && !(low > 0.0))))
        return SV_ERR_INVALID_ARG;
    const double r = rotary_dim, two_pi = 6.283185307179586476925;
    if (scaling == SV_ROPE_SCALE_BASE) base *= pow(factor, r / (r - 2.0));
    double d_high = 0.0, d_low = 0.0;
    if (scaling == SV_ROPE_SCALE_DIMS) {
        auto dim_of = [&](double turns) { return r * log((double)original_len / (two_pi * turns)) / (2.0 * log(base)); };
        d_high = fmin(fmax(floor(dim_of(high)), 0.0), r - 1.0);
        d_low = fmin(fmax(ceil(dim_of(low)), 0.0), r - 1.0);
        if (d_low - d_high < 0.001) d_low = d_high + 0.001;
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / r);
        if (scaling == SV_ROPE_SCALE_LINEAR) {
            f /= factor;
        } else if (scaling == SV_ROPE_SCALE_TURNS) {
            const double g = fmin(fmax(((double)original_len * f / two_pi - low) / (high - low), 0.0), 1.0);
            f *= g + (1.0 - g) / factor;
        } else if (scaling == SV_ROPE_SCALE_DIMS) {
            const double h = fmin(fmax((i - d_high) / (d_low - d_high), 0.0), 1.0);
            f *= 1.0 - h + h / factor;
        }
        inv_freq[i] = (float)f;
    }
    *magnitude = scaling == SV_ROPE_SCALE_DIMS ? (float)(1.0 + 0.1 * log(factor)) : 1.0f;
    return SV_OK;
}

static bool rope_ok(const float *inv_freq, int rotary_dim, int style, int head_dim) {
    if (style != SV_ROPE_HALF && style != SV_ROPE_INTERLEAVED) return false;
    if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > head_dim || rotary_dim > SV_KV_MAX_HEAD_DIM) return false;
    return rotary_dim == 0 || inv_freq != nullptr;
}

// A rotation in place is fine, one onto other rows that are still read is not.
static bool turns_onto(const RowsView &x, const RowsView &out) { return !same_place(x, out) && overlap(x, out); }

extern "C" sv_status sv_rope(const void *x, int64_t x_row_stride, int64_t x_head_stride, void *out,
                             int64_t out_row_stride, int64_t out_head_stride, sv_dtype dtype, int64_t rows, int heads,
                             int head_dim, const int32_t *positions, const float *inv_freq, int rotary_dim, int style,
                             float magnitude, int backward, sv_stream_t stream) {
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
    if (rows < 0 || rows > INT32_MAX || heads < 1 || head_dim < 1 || rotary_dim < 2 ||
        !rope_ok(inv_freq, rotary_dim, style, head_dim) || (int64_t)heads * head_dim > INT32_MAX)
        return SV_ERR_INVALID_ARG;
    if (rows == 0) return SV_OK;
    if (x == nullptr || out == nullptr || positions == nullptr) return SV_ERR_INVALID_ARG;
    const int es = elem_size(dtype);
    if (turns_onto({x, x_row_stride * es, x_head_stride * es, rows, heads, (int64_t)head_dim * es},
                   {out, out_row_stride * es, out_head_stride * es, rows, heads, (int64_t)head_dim * es}))
        return SV_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on_current_device(s, x, out)) return SV_ERR_INVALID_ARG;
    RopeArgs a{static_cast<const char *>(x), static_cast<char *>(out), x_row_stride * es, x_head_stride * es,
               out_row_stride * es, out_head_stride * es, positions, inv_freq, {heads, head_dim, rotary_dim / 2, style},
               magnitude, backward ? -1.0f : 1.0f};
    // Vectors where every one of them starts on 16 bytes, single elements otherwise.
    const bool vec = rot_vec(rotary_dim / 2, style, es) && (head_dim * es) % 16 == 0 && aligned(x, 16) && aligned(out, 16) &&
                     strides16(es, x_row_stride, x_head_stride) && strides16(es, out_row_stride, out_head_stride);
    const dim3 grid((unsigned)rows);
    if (es == 4)
        vec ? k_rope<4, true><<<grid, kRopeThreads, 0, s>>>(a) : k_rope<4, false><<<grid, kRopeThreads, 0, s>>>(a);
    else
        vec ? k_rope<2, true><<<grid, kRopeThreads, 0, s>>>(a) : k_rope<2, false><<<grid, kRopeThreads, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}

extern "C" sv_status sv_kv_append(const sv_kv_cache *cache, const sv_kv_batch *batch, const void *q,
                                  int64_t q_row_stride, int64_t q_head_stride, void *q_out, int64_t q_out_row_stride,
                                  int64_t q_out_head_stride, int q_heads, const void *k, int64_t k_row_stride,
                                  int64_t k_head_stride, const void *v, int64_t v_row_stride, int64_t v_head_stride,
                                  const float *inv_freq, int rotary_dim, int style, float magnitude, sv_stats *stats,
                                  sv_stream_t stream) {
    if (!kv_args_ok(cache, batch, true) || !rope_ok(inv_freq, rotary_dim, style, cache->head_dim))
        return SV_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (q != nullptr && q_heads < 1)) return SV_ERR_INVALID_ARG;
    const int es = elem_size((sv_dtype)cache->dtype);
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on_current_device(s, cache->k, k)) return SV_ERR_INVALID_ARG;
    if (stats && cudaMemsetAsync(stats, 0, sizeof(sv_stats), s) != cudaSuccess) return SV_ERR_CUDA;
    AppendArgs a{kv_cache_of(*cache), kv_batch_of(*batch), static_cast<const char *>(q), static_cast<const char *>(k),
                 static_cast<const char *>(v), static_cast<char *>(q_out), q_row_stride * es, q_head_stride * es,
                 q_out_row_stride * es, q_out_head_stride * es, k_row_stride * es, k_head_stride * es, v_row_stride * es,
                 v_head_stride * es, inv_freq, {q_heads, cache->head_dim, rotary_dim / 2, style}, magnitude, stats};
    const bool vec = rot_vec(rotary_dim / 2, style, es);
    if (batch->rows == 0) return SV_OK;
    const dim3 grid((unsigned)batch->rows);
    if (es == 4)
        vec ? k_kv_append<4, true><<<grid, kRopeThreads, 0, s>>>(a) : k_kv_append<4, false><<<grid, kRopeThreads, 0, s>>>(a);
    else
        vec ? k_kv_append<2, true><<<grid, kRopeThreads, 0, s>>>(a) : k_kv_append<2, false><<<grid, kRopeThreads, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}

extern "C" sv_status sv_kv_commit(const sv_kv_cache *cache, const sv_kv_batch *batch, int n_layers,
                                  int64_t layer_stride, const int32_t *accept_len, const int32_t *path,
                                  int32_t *context_out, sv_stats *stats, sv_stream_t stream) {
    if (!kv_args_ok(cache, batch, false) || n_layers < 1 || accept_len == nullptr || batch->n - 1 > SV_MAX_TREE ||
        (path == nullptr && batch->n > 1) || context_out == batch->context_len)
        return SV_ERR_INVALID_ARG;
    const int es = elem_size((sv_dtype)cache->dtype);
    if (!strides16(es, layer_stride) || (int64_t)batch->B * n_layers > INT32_MAX) return SV_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!on_current_device(s, cache->k, accept_len)) return SV_ERR_INVALID_ARG;
    if (stats && cudaMemsetAsync(stats, 0, sizeof(sv_stats), s) != cudaSuccess) return SV_ERR_CUDA;
    CommitArgs a{kv_cache_of(*cache), kv_batch_of(*batch), layer_stride * es, accept_len, path, context_out, stats};
    k_kv_commit<<<(unsigned)(batch->B * n_layers), 256, 0, s>>>(a, es);
    return cuda_status(cudaGetLastError());
}
