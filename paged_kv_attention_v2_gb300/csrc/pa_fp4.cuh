// pa_fp4.cuh -- 4-bit pages: e2m1 codes and e4m3 scales to fp16.
#pragma once

#include <stdint.h>

namespace pa {

// Eight e2m1 codes (the lowest bits first) as four f16x2 pairs (exact).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// The two e4m3 codes in the low half of w as an f16x2 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(h) : "r"(w));
    return h;
}

// A bf16x2 pair as f16x2, beyond 65504: that number.
__device__ __forceinline__ uint32_t bf16x2_to_f16(uint32_t w) {
    uint32_t d;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(__uint_as_float(w & 0xffff0000u)), "f"(__uint_as_float(w << 16)));
    return d;
}

// The larger magnitude of two f16x2 pairs, element by element (of NaN and a number the number).
__device__ __forceinline__ uint32_t max_magnitude_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("{\n\t.reg .b32 x, y;\n\tabs.f16x2 x, %1;\n\tabs.f16x2 y, %2;\n\tmax.f16x2 %0, x, y;\n\t}" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Products of f16x2 pairs (a code times a scale: at most six significant bits, between
// 2^-10 and 2688, so exact).
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Even codes of a and b in one word, odd ones in another: byte i of `even` holds code 2i
// of a (low half) and of b, byte i of `odd` code 2i + 1 of both.
__device__ __forceinline__ void pair_codes(uint32_t a, uint32_t b, uint32_t& even, uint32_t& odd) {
    even = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
    odd = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
}

}  // namespace pa
