// sv_code8.cuh — the cache held in 8 bits: e4m3 codes, their power-of-two scales, and the moves between codes, float32 and bf16.
#pragma once

#include <cuda_fp16.h>

#include "sv_kv.cuh"

namespace sv {

// Scales of a cache held in 8 bits (null pointers: none).  Byte strides.
struct KvScale {
    const uint8_t *k, *v;
    int64_t page_b, head_b;
};

constexpr int kScaleLowest = 7;   // least byte an append writes: every code's value is then a bf16 number

inline KvCache kv_cache_of(const sv_kv_cache8 &c) {
    return {static_cast<char *>(c.k), static_cast<char *>(c.v), c.page_stride, c.slot_stride, c.head_stride, c.n_pages, c.page_size, c.kv_heads,
            c.head_dim};
}
inline KvScale kv_scale_of(const sv_kv_cache8 &c) { return {c.k_scale, c.v_scale, c.scale_page_stride, c.scale_head_stride}; }

// The checks of kv_args_ok; the codes' strides are bytes.
inline bool kv_args_ok(const sv_kv_cache8 *c, const sv_kv_batch *b, sv_dtype dtype, bool block) {
    if (c == nullptr || c->k_scale == nullptr || c->v_scale == nullptr || (dtype != SV_F32 && dtype != SV_BF16)) return false;
    if (c->page_stride % 16 != 0 || c->slot_stride % 16 != 0 || c->head_stride % 16 != 0 || c->head_dim % 16 != 0) return false;
    const sv_kv_cache as{c->k, c->v, c->page_stride, c->slot_stride, c->head_stride, c->n_pages, c->page_size, c->kv_heads, c->head_dim, dtype};
    return kv_args_ok(&as, b, block);
}

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FFFFFFFu : byte << 23);
}

// The byte of the smallest scale, kScaleLowest at least, that keeps `most` (finite, >= 0) within 448 = 1.75 * 2^8: with most = f 2^E it is
// E - 8, one more where f > 1.75, which adding 0x1FFFFF to the fraction's bits carries into the exponent's.
__device__ __forceinline__ int scale_for(float most) {
    return max((int)((__float_as_uint(most) + 0x1FFFFFu) >> 23) - 8, kScaleLowest);
}

// Two codes (the first in the low byte) as floats.
__device__ __forceinline__ float2 codes2(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ float4 codes4(uint32_t four) {
    const float2 a = codes2(four), b = codes2(four >> 16);
    return make_float4(a.x, a.y, b.x, b.y);
}

// Four codes as two pairs of binary16 numbers.
__device__ __forceinline__ void codes4_f16(uint32_t four, uint32_t &a, uint32_t &b) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(four));
}

// Two floats of at most 448 as codes, to nearest, ties to even; NaN stays NaN.
__device__ __forceinline__ uint32_t to_codes2(float lo, float hi) {
    uint32_t two;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %1, %2;\n\tcvt.u32.u16 %0, c;\n\t}" : "=r"(two) : "f"(hi), "f"(lo));
    return two;
}

// Four codes in a scale 2^shift times theirs.  Binary16 holds what a code that does not become 0 turns into exactly: the only
// rounding is that to the code.
__device__ __forceinline__ uint32_t rescaled4(uint32_t four, __half2 factor) {
    uint32_t out;
    asm("{\n\t.reg .b16 a, b;\n\t.reg .b32 x, y;\n\t"
        "mov.b32 {a, b}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 x, a;\n\tcvt.rn.f16x2.e4m3x2 y, b;\n\t"
        "mul.rn.f16x2 x, x, %2;\n\tmul.rn.f16x2 y, y, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, x;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, y;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(out)
        : "r"(four), "r"(*reinterpret_cast<const uint32_t *>(&factor)));
    return out;
}
// 2^-shift; from 2^-24 on every code but NaN becomes 0 either way.
__device__ __forceinline__ __half2 rescale_factor(int shift) {
    return __half2half2(__float2half_rn(__uint_as_float((uint32_t)(127 - min(shift, 24)) << 23)));
}
__device__ __forceinline__ uint4 rescaled16(uint4 w, int shift) {
    if (shift == 0) return w;
    const __half2 f = rescale_factor(shift);
    return make_uint4(rescaled4(w.x, f), rescaled4(w.y, f), rescaled4(w.z, f), rescaled4(w.w, f));
}

}  // namespace sv
