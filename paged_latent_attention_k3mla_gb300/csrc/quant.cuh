// quant.cuh -- the 8-bit latent cache's rows.
//
// A token's row in a layer is 512 e4m3 codes, 64 bf16 rope entries and a power of two 2^n as a bf16; it stands for the latent
// code_j 2^n and the rope key rope_i 2^n.  n is the smallest that brings the row's largest finite latent m to 448, e4m3's
// largest, or below: m = f 2^e with f in [1/2, 1) gives n = e - 9, one more where f > 7/8.  One scale a row, and a power of
// two: e4m3 has an exponent of its own, so entries down to 2^-6 / 448 of the largest keep their 4 bits under any scale, and
// scaling by a power of two rounds nothing -- the code is one rounding of c 2^-n, and what is read back is exact in bf16.
// The rope key is kept in units of the same power of two (exact, but for entries below 2^(n - 126)), so that both parts of a
// score, and the tensor core's sum of them, have one factor.  For that n is also large enough to keep the rope entries below
// 2^120, and lies in [-96, 120]: rows whose largest latent is below 2^-88 lose bits to e4m3's smallest step.
// NaN and infinities among the latents become the NaN code and do not count for n.
//
// A page of a layer is one block: 64 rows of 640 bytes (whole 128-byte lines), then 64 scales: 41,088 B, 642 a token.
#pragma once
#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace k3 {

constexpr int QROW = K3MLA_QUANT_ROW_BYTES;             // 640
constexpr int QPAGE = K3MLA_QUANT_PAGE_BYTES;           // 41,088
constexpr int QSCALES = PAGE * QROW;                    // where a page's scales begin
static_assert(QROW == LORA + 2 * ROPE && QPAGE == QSCALES + 2 * PAGE && QPAGE % 128 == 0, "whole lines");

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8])
{
    x[0] = bf16lo_to_f32(v.x), x[1] = bf16hi_to_f32(v.x);
    x[2] = bf16lo_to_f32(v.y), x[3] = bf16hi_to_f32(v.y);
    x[4] = bf16lo_to_f32(v.z), x[5] = bf16hi_to_f32(v.z);
    x[6] = bf16lo_to_f32(v.w), x[7] = bf16hi_to_f32(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Two e4m3 codes (lo in bits 0..7), round to nearest even; larger ones become 448, NaN the NaN code.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (bits 0..15) as a pair of f16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}

// A pair of f16 as codes, likewise.
__device__ __forceinline__ uint32_t pack_e4m3x2_f16(uint32_t v)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
    return r;
}

// 2^13 (v - part) of two pairs of f16, exact where part is v rounded to e4m3's bits.
__device__ __forceinline__ uint32_t rest_f16x2(uint32_t v, uint32_t part)
{
    uint32_t d;
    asm("{\n\t.reg .b32 s;\n\tmov.b32 s, 0x70007000;\n\tsub.rn.f16x2 %0, %1, %2;\n\tmul.rn.f16x2 %0, %0, s;\n\t}" : "=&r"(d) : "r"(v), "r"(part));
    return d;
}

// Eight e4m3 codes as f32, exact.
__device__ __forceinline__ void e4m3x8_to_f32(const uint2& v, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f16x2_parts(e4m3x2_to_f16x2(((i & 2) ? v.y : v.x) >> (16 * (i & 1))), x[2 * i], x[2 * i + 1]);
}

// The largest magnitude among eight, as bits (they order like the magnitudes); NaN and infinities count as 0 and set `odd`.
__device__ __forceinline__ uint32_t largest_finite(const float (&x)[8], bool& odd)
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(x[e]) & 0x7FFFFFFFu;
        if (b >= 0x7F800000u) odd = true;
        else m = max(m, b);
    }
    return m;
}

// n for a row whose largest finite latent and rope entry have the bits m and r (of f32, without signs).
__device__ __forceinline__ int quant_exponent(uint32_t m, uint32_t r)
{
    // (the exponent fields are e + 126)
    const int n = m ? (int)(m >> 23) - 135 + ((m & 0x7FFFFFu) > 0x600000u) : 0;
    return min(max(max(n, (int)(r >> 23) - 246), -96), 120);
}

// A row into its place in a page block, by a whole warp: lane l has the latents 8 l .. and 256 + 8 l .., and lanes 0 .. 7 the
// rope entries 8 l .. (the others' k is not looked at).  `block`: the page's block of the layer, line the row in it.
__device__ __forceinline__ void quant_store_row(uint8_t* block, int line, float (&c0)[8], float (&c1)[8], const float (&k)[8])
{
    const int lane = (int)lane_id();
    bool odd = false, rope_odd = false;
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(largest_finite(c0, odd), largest_finite(c1, odd)));
    const uint32_t r = __reduce_max_sync(0xFFFFFFFFu, lane < 8 ? largest_finite(k, rope_odd) : 0u);
    const int n = quant_exponent(m, r);
    const float down = __uint_as_float((uint32_t)(127 - n) << 23);
    if (__any_sync(0xFFFFFFFFu, odd)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if ((__float_as_uint(c0[e]) & 0x7F800000u) == 0x7F800000u) c0[e] = __uint_as_float(0x7FFFFFFFu);
            if ((__float_as_uint(c1[e]) & 0x7F800000u) == 0x7F800000u) c1[e] = __uint_as_float(0x7FFFFFFFu);
        }
    }
    auto codes = [&](const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_e4m3x2(x[2 * i] * down, x[2 * i + 1] * down);
        return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    };
    uint8_t* row = block + line * QROW;
    *reinterpret_cast<uint2*>(row + 8 * lane) = codes(c0);
    *reinterpret_cast<uint2*>(row + 256 + 8 * lane) = codes(c1);
    if (lane < 8) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = k[e] * down;
        *reinterpret_cast<uint4*>(row + LORA + 16 * lane) = pack8(y);
    }
    if (lane == 0) *reinterpret_cast<uint16_t*>(block + QSCALES + 2 * line) = (uint16_t)((n + 127) << 7);
}

}  // namespace k3
