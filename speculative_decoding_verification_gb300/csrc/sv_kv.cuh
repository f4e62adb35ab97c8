// sv_kv.cuh — shared by the kernels of the target's side of a step: the paged cache's addresses, the
// block's rows and depths, and the rotation of a position's pairs.
#pragma once

#include <utility>

#include "sv_device.cuh"
#include "sv_host.h"

namespace sv {

// A cache as the kernels read it: byte strides, element size folded in.
struct KvCache {
    char *k, *v;
    int64_t page_b, slot_b, head_b;
    int n_pages, page_size, kv_heads, head_dim;
};

struct KvBatch {
    const int32_t *context_len, *page_table, *row_start, *parents;
    int64_t table_pitch;
    int max_pages, B, n, rows;
};

inline KvCache kv_cache_of(const sv_kv_cache &c) {
    const int es = elem_size((sv_dtype)c.dtype);
    return {static_cast<char *>(c.k), static_cast<char *>(c.v), c.page_stride * es, c.slot_stride * es, c.head_stride * es,
            c.n_pages, c.page_size, c.kv_heads, c.head_dim};
}

inline KvBatch kv_batch_of(const sv_kv_batch &b) {
    return {b.context_len, b.page_table, b.row_start, b.parents, b.table_pitch, b.max_pages, b.B, b.n, b.rows};
}

// Strides and bases that 16-byte vectors can be used with.
inline bool strides16(int es, int64_t a, int64_t b = 0, int64_t c = 0) {
    return (a * es) % 16 == 0 && (b * es) % 16 == 0 && (c * es) % 16 == 0;
}

// Most slots of a page table: places up to a few tiles past the last slot are formed in 32 bits.
constexpr int64_t kMaxSlots = INT32_MAX - 1024;

// An array [rows][heads] of `width` bytes each, strides in bytes.
struct RowsView {
    const void *base;
    int64_t row, head, rows, heads, width;
};

inline bool same_place(const RowsView &a, const RowsView &b) {
    return a.base == b.base && (a.rows <= 1 || a.row == b.row) && (a.heads <= 1 || a.head == b.head);
}

// Whether some byte belongs to both.  Exact for arrays of one row stride (views of one projection interleave without sharing); of arrays
// with different row strides, or of thousands of heads with different head strides, only those that start at one address are said to.
inline bool overlap(RowsView a, RowsView b) {
    if (a.rows < 1 || b.rows < 1) return false;
    if (a.base == b.base) return true;
    auto low = [](const RowsView &v) { return (v.row < 0 ? (v.rows - 1) * v.row : 0) + (v.head < 0 ? (v.heads - 1) * v.head : 0); };
    auto high = [](const RowsView &v) { return (v.row > 0 ? (v.rows - 1) * v.row : 0) + (v.head > 0 ? (v.heads - 1) * v.head : 0) + v.width; };
    const int64_t d = (int64_t)((intptr_t)b.base - (intptr_t)a.base);   // b from a
    if (high(a) <= d + low(b) || d + high(b) <= low(a)) return false;
    if (a.rows == 1) a.row = b.row;
    if (b.rows == 1) b.row = a.row;
    if (a.row != b.row) return false;
    const bool one = a.head == b.head;
    if (one && a.heads + b.heads > a.rows + b.rows) {   // rows and heads are alike: the longer axis is solved for, the shorter walked
        std::swap(a.row, a.head);
        std::swap(a.rows, a.heads);
        std::swap(b.row, b.head);
        std::swap(b.rows, b.heads);
    }
    if (!one && a.heads * b.heads > 1 << 20) return false;
    // Row r of a and row r + s of b, -a.rows < s < b.rows, are s row strides apart: looks for the s that brings two heads nearest.
    auto meets = [&](int64_t apart) {   // b's head from a's, in one row
        if (a.row == 0) return apart < b.width && -apart < a.width;
        const int64_t q = -apart / a.row;
        for (int64_t s = q - 1; s <= q + 1; ++s) {
            const int64_t in = s < 1 - a.rows ? 1 - a.rows : s > b.rows - 1 ? b.rows - 1 : s, x = apart + in * a.row;
            if (x < b.width && -x < a.width) return true;
        }
        return false;
    };
    for (int64_t i = 0; i < (one ? 1 : a.heads); ++i)   // with one head stride only the heads' difference counts
        for (int64_t j = one ? 1 - a.heads : 0; j < b.heads; ++j)
            if (meets(d + j * b.head - i * a.head)) return true;
    return false;
}

inline bool kv_args_ok(const sv_kv_cache *c, const sv_kv_batch *b, bool block) {
    if (c == nullptr || b == nullptr || c->k == nullptr || c->v == nullptr) return false;
    if (c->dtype != SV_F32 && c->dtype != SV_BF16) return false;
    const int es = elem_size((sv_dtype)c->dtype);
    if (c->n_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1 || c->head_dim > SV_KV_MAX_HEAD_DIM)
        return false;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !strides16(es, c->page_stride, c->slot_stride, c->head_stride) ||
        !strides16(es, c->head_dim))
        return false;
    if (b->context_len == nullptr || b->page_table == nullptr || b->B < 1 || b->n < 1 || b->max_pages < 1 ||
        b->table_pitch < b->max_pages)
        return false;
    if ((int64_t)b->max_pages * c->page_size > kMaxSlots || (b->row_start == nullptr && (int64_t)b->B * b->n > INT32_MAX))
        return false;
    if (block) {
        if (b->rows < 0 || (b->row_start == nullptr && b->rows != b->B * b->n)) return false;
        if (b->parents != nullptr && (b->row_start != nullptr || b->n - 1 > SV_MAX_TREE)) return false;
    }
    return true;
}

inline bool rope_args_ok(const float *inv_freq, int rotary_dim, int style, int head_dim) {
    if (style != SV_ROPE_HALF && style != SV_ROPE_INTERLEAVED) return false;
    if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > head_dim || rotary_dim > SV_KV_MAX_HEAD_DIM) return false;
    return rotary_dim == 0 || inv_freq != nullptr;
}

// A rotation in place is fine, one onto other rows that are still read is not.
inline bool turns_onto(const RowsView &x, const RowsView &out) { return !same_place(x, out) && overlap(x, out); }

// Rows [r0, r0 + n) of sequence b; a row_start that falls, passes `rows` or holds more than n rows gives
// none (ok = false).
struct SeqRows {
    int r0, n;
    bool ok;
};

__host__ __device__ __forceinline__ SeqRows seq_rows(const KvBatch &bt, int b) {
    if (bt.row_start == nullptr) return {b * bt.n, bt.n, true};
    const int r0 = bt.row_start[b], r1 = bt.row_start[b + 1];
    if (r0 < 0 || r1 < r0 || r1 > bt.rows || r1 - r0 > bt.n) return {0, 0, false};
    return {r0, r1 - r0, true};
}

// The sequence of a row: the last b with row_start[b] <= row (a row of none gives some b without it).
__device__ __forceinline__ int row_sequence(const KvBatch &bt, int row) {
    if (bt.row_start == nullptr) return row / bt.n;
    int lo = 0, hi = bt.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (bt.row_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Byte offset of slot s of the sequence whose page table row is `table` (head 0), or -1 for a bad page id.
__device__ __forceinline__ int64_t slot_offset(const KvCache &c, const int32_t *table, int s) {
    const int p = s / c.page_size;
    const int page = table[p];
    if (page < 0 || page >= c.n_pages) return -1;
    return page * c.page_b + (s - p * c.page_size) * c.slot_b;
}

// ------------------------------------------------------------------------------------------
// Rotation
// ------------------------------------------------------------------------------------------
// cos and sin of t * f for an int32 position t.  The angle is formed in turns as an unevaluated
// sum: g = f / 2pi to about 47 bits, t = th + tl exactly, p = th * g.hi with its rounding error, and
// whole turns are dropped before the parts are added.  A float32 product t * f would be off by
// 2^-25 t f rad, 4e-3 at t = 131072; this one stays within 2e-6 + 1.5e-14 |t|.
__device__ __forceinline__ float2 rope_cos_sin(int t, float f) {
    constexpr float I_HI = 0x1.45f306p-3f, I_LO = 0x1.b9391p-28f;   // 1 / 2pi
    ff g = two_prod(f, I_HI);
    g.lo = __fmaf_rn(f, I_LO, g.lo);
    const float th = (float)t;
    const float tl = (float)(t - (int)fminf(th, 2147483520.0f));   // |t - th| <= 127: exact
    const float thc = fminf(th, 2147483520.0f);
    const ff p = two_prod(thc, g.hi);
    float turn = __fsub_rn(p.hi, rintf(p.hi));
    turn += __fsub_rn(p.lo, rintf(p.lo)) + __fmaf_rn(thc, g.lo, __fmul_rn(tl, g.hi));
    turn -= rintf(turn);
    float s, c;
    sincospif(2.0f * turn, &s, &c);
    return make_float2(c, s);
}

template <int ES>
__device__ __forceinline__ uint4 pack16(const float (&x)[16 / ES]) {
    if constexpr (ES == 4) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int ES>
__device__ __forceinline__ void store_elem(char *p, float x) {
    if constexpr (ES == 4) {
        *reinterpret_cast<float *>(p) = x;
    } else {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
        *reinterpret_cast<uint16_t *>(p) = h;
    }
}

// Rotates the heads of one row.  cs[i] = (cos, sin) of pair i, the magnitude and the direction folded in.  Item i of
// the row is a 16-byte vector (VEC; in the half style the two vectors whose elements pair up) or one
// pair / one copied element.  One thread takes both sides of a pair, so out may be x.
struct RotShape {
    int heads, dim, half;   // half = rotary_dim / 2
    int style;
};

template <int ES, bool VEC>
__device__ __forceinline__ int rot_items(const RotShape &s) {
    constexpr int E = VEC ? 16 / ES : 1;
    const int turned = s.half == 0 ? 0 : VEC && s.style == SV_ROPE_INTERLEAVED ? 2 * s.half / E : s.half / E;
    return turned + (s.dim - 2 * s.half) / E;   // items of one head
}

template <int ES, bool VEC>
__device__ __forceinline__ void rot_item(const RotShape &s, const char *x, char *out, int i, const float2 *cs) {
    if constexpr (VEC) {
        constexpr int E = 16 / ES;
        const bool inter = s.style == SV_ROPE_INTERLEAVED;
        const int turned = inter ? 2 * s.half / E : s.half / E;
        if (i >= turned) {
            const int e = 2 * s.half + (i - turned) * E;
            *reinterpret_cast<uint4 *>(out + (size_t)e * ES) = *reinterpret_cast<const uint4 *>(x + (size_t)e * ES);
            return;
        }
        float a[E];
        if (inter) {
            const int e = i * E;
            unpack<ES>(*reinterpret_cast<const uint4 *>(x + (size_t)e * ES), a);
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float2 c = cs[e / 2 + j];
                const float u = a[2 * j], w = a[2 * j + 1];
                a[2 * j] = __fmaf_rn(u, c.x, -__fmul_rn(w, c.y));
                a[2 * j + 1] = __fmaf_rn(u, c.y, __fmul_rn(w, c.x));
            }
            *reinterpret_cast<uint4 *>(out + (size_t)e * ES) = pack16<ES>(a);
        } else {
            const int e = i * E;
            float b[E];
            unpack<ES>(*reinterpret_cast<const uint4 *>(x + (size_t)e * ES), a);
            unpack<ES>(*reinterpret_cast<const uint4 *>(x + (size_t)(e + s.half) * ES), b);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float2 c = cs[e + j];
                const float u = a[j], w = b[j];
                a[j] = __fmaf_rn(u, c.x, -__fmul_rn(w, c.y));
                b[j] = __fmaf_rn(u, c.y, __fmul_rn(w, c.x));
            }
            *reinterpret_cast<uint4 *>(out + (size_t)e * ES) = pack16<ES>(a);
            *reinterpret_cast<uint4 *>(out + (size_t)(e + s.half) * ES) = pack16<ES>(b);
        }
    } else {
        if (i >= s.half) {
            const size_t e = (size_t)(s.half + i) * ES;   // 2 half + (i - half)
            if constexpr (ES == 4) *reinterpret_cast<uint32_t *>(out + e) = *reinterpret_cast<const uint32_t *>(x + e);
            else *reinterpret_cast<uint16_t *>(out + e) = *reinterpret_cast<const uint16_t *>(x + e);
            return;
        }
        const int e0 = s.style == SV_ROPE_INTERLEAVED ? 2 * i : i;
        const int e1 = s.style == SV_ROPE_INTERLEAVED ? 2 * i + 1 : i + s.half;
        const float2 c = cs[i];
        float u, w;
        if constexpr (ES == 4) {
            u = reinterpret_cast<const float *>(x)[e0];
            w = reinterpret_cast<const float *>(x)[e1];
        } else {
            u = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(x)[e0] << 16);
            w = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(x)[e1] << 16);
        }
        store_elem<ES>(out + (size_t)e0 * ES, __fmaf_rn(u, c.x, -__fmul_rn(w, c.y)));
        store_elem<ES>(out + (size_t)e1 * ES, __fmaf_rn(u, c.y, __fmul_rn(w, c.x)));
    }
}

// Whether a head's rotated part splits into whole 16-byte vectors.
inline bool rot_vec(int half, int style, int es) {
    return style == SV_ROPE_INTERLEAVED ? (2 * half * es) % 16 == 0 : (half * es) % 16 == 0;
}

}  // namespace sv
