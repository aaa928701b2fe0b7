// rows8.cuh -- the 8-bit row format of the norm's output and of the layer's
// saved training state: E4M3 values with one power-of-two scale per block of
// 32 consecutive columns of a row (the last block of a row may be shorter).
//
// With a = the largest finite |v| of a block, its exponent is
//   e = the smallest integer with a <= 448 * 2^e, held to [-124, 120],
// stored as the byte e + 127, and a value is stored as rn_e4m3(v * 2^-e),
// ties to even. 448 is the largest E4M3 value, so nothing saturates; fp32
// values reach 2^128, hence 120 (where values are held to 240 * 2^120, the
// largest that bf16 holds). The product v * 2^-e is exact in fp32, so a
// value is rounded once. A value read back, (E4M3 value) * 2^e, has four
// significant bits and is at least 2^-9 * 2^-124 = 2^-133, the smallest bf16:
// bf16 holds it exactly, so it feeds bf16 tensor cores without a second
// rounding. An infinity or NaN is stored as NaN and leaves the rest of its
// block as it would be without it.
#pragma once

#include <cuda_fp8.h>

#include "moe_common.cuh"

namespace moe {

constexpr int kRows8Block = 32;

__host__ __device__ constexpr int rows8_blocks(int cols) { return (cols + kRows8Block - 1) / kRows8Block; }

// The scale byte of a block whose largest finite magnitude is a (>= 0, finite).
// With a = m * 2^E, 1 <= m < 2: e = E - 8 if m <= 1.75, else E - 7; adding
// 0x1FFFFF to the bits carries into the exponent field exactly when m > 1.75.
__device__ __forceinline__ uint32_t rows8_scale_byte(float a) {
    const int field = (int)((__float_as_uint(a) + 0x1FFFFFu) >> 23);   // biased E (+ 1)
    return (uint32_t)max(field - 8, 3);                                // e + 127; at most 247 for a finite a
}

// 2^-e and 2^e of a scale byte e + 127 (the library writes bytes 3..247).
__device__ __forceinline__ float rows8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float rows8_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// A block whose largest magnitude (NaN left out) reaches this holds infinities or
// has e = 120, the two cases that rows8_scaled_special and rows8_finite are for.
constexpr float kRows8Special = 0x1.cp+127f;   // 448 * 2^119

// |v| of a finite v, else 0: what counts towards a block's scale.
__device__ __forceinline__ float rows8_finite(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.0f;
}

// v * 2^-e in a special block: an infinity becomes NaN, and at e = 120 the
// magnitude is held to 240, since 256 * 2^120 is past fp32 and bf16.
__device__ __forceinline__ float rows8_scaled_special(float v, uint32_t byte) {
    if (!(fabsf(v) < INFINITY)) return NAN;
    const float s = v * rows8_inv_scale(byte);
    if (byte != 247u) return s;
    return s > 240.0f ? 240.0f : s < -240.0f ? -240.0f : s;
}

// Two values as E4M3, the first in the low byte.
__device__ __forceinline__ uint32_t rows8_pack2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Four values as E4M3, the first in the lowest byte.
__device__ __forceinline__ uint32_t rows8_pack4(float a, float b, float c, float d) {
    return rows8_pack2(a, b) | (rows8_pack2(c, d) << 16);
}

// The two E4M3 values in the low 16 bits of w, unscaled.
__device__ __forceinline__ float2 rows8_unpack2(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    return __half22float2(__half2(h));
}

// Stores a thread's eight columns of a block that four adjacent lanes share
// (lane & ~3 .. + 3, each with eight columns in order; absent columns hold 0):
// the lanes agree on the block's scale, each packs its columns, and the caller
// stores q and (one lane of the four) the returned byte. All lanes of the warp
// must call it together.
__device__ __forceinline__ uint32_t rows8_quantize_quad(const float (&v)[8], uint2& q) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));   // a NaN does not count
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
    uint32_t byte = rows8_scale_byte(a);
    float s[8];
    if (__any_sync(0xFFFFFFFFu, a >= kRows8Special)) {
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fmaxf(a, rows8_finite(v[i]));
        a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
        byte = rows8_scale_byte(a);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = rows8_scaled_special(v[i], byte);
    } else {
        const float inv = rows8_inv_scale(byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = v[i] * inv;
    }
    q = make_uint2(rows8_pack4(s[0], s[1], s[2], s[3]), rows8_pack4(s[4], s[5], s[6], s[7]));
    return byte;
}

// Eight values read back, as bf16 pairs (exact).
__device__ __forceinline__ uint4 rows8_dequantize8(uint2 q, uint32_t byte) {
    const float s = rows8_scale(byte);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = rows8_unpack2((i < 2 ? q.x : q.y) >> (16 * (i & 1)));
        w[i] = pack_bf16x2(f.x * s, f.y * s);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace moe
