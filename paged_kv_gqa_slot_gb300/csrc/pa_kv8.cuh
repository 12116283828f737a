// pa_kv8.cuh -- the 8-bit pool's number format on the device, shared by the kernels that
// write it (pa_append8.cu) and read it (pa_decode_lanes.cu, pa_prefill8.cu).
//
// A (block, kv head) tile of K or of V holds e4m3 codes and one power-of-two scale:
//     value = e4m3(code) * 2^k,   k = exps[block, kv head, 0 (K) or 1 (V)] - 127.
// Powers of two because e4m3 is a floating-point format: the scale only has to bring the
// tile's largest magnitude under 448, and a finer scale would buy no precision (but for e4m3's
// subnormals).  In return every step but the one rounding to e4m3 is exact: x / 2^k, the
// product code * 2^k (a bf16 number), and the shift of a tile's codes to a larger scale.
#pragma once

#include <cuda_fp16.h>

#include "pa_device.cuh"

namespace pa {

// k of a stored exponent, and its range: 448 * 2^119 is the largest such product below the
// bf16 (and fp32) maximum, and 2^-9 * 2^-100 keeps every code's value a normal bf16 number.
constexpr int kExpBias = 127;
constexpr int kExpMin = -100, kExpMax = 119;

// 2^e for -126 <= e <= 127 (clamped to that range)
__device__ __forceinline__ float exp2_int(int e) {
    return __int_as_float((min(max(e, -126), 127) + 127) << 23);
}

// An exponent byte brought into the range the format has: a tile that was never written may hold
// anything, zeros first of all.  And a block's word of them (K in the low byte).
__device__ __forceinline__ int valid_exp(int byte) { return min(max(byte, kExpMin + kExpBias), kExpMax + kExpBias); }
__device__ __forceinline__ int valid_exps(int word) { return valid_exp(word & 255) | valid_exp(word >> 8 & 255) << 8; }

// The kernels' softmax weighs V by u = 2^(x + kV - base) (but for a constant factor) and sums the normaliser's 2^(x - base) as u 2^-kV.
// u ends at 2^-126 and the normaliser holds 2^-kB of the block that set the base, so that is right as
// long as kB - kV stays far below 126: with every kV a row has seen within +-kNearScale, terms below
// 2^(96 - 126) of the normaliser are lost.  From the first V exponent byte outside on, the terms
// are taken by an exponential of their own.
constexpr int kNearScale = 48;

// u is rounded to f16, which has 11 bits from 2^-14 on and ends at 2^16 and 2^-25.  A base kHeadroom log2
// units below the row's maximum uses f16's upper range, so that u keeps its bits down to 2^-21 of the
// largest and some down to 2^-32: with one key that takes 0.9998 of a row and has no value of its own, the rest
// over 4095 others, the result is right to 2^-8 (with the base at the maximum it was 5% off).  The normaliser
// takes u 2^(-kV - kHeadroom), a normal factor for every kV.
constexpr int kHeadroom = 7;
__device__ __forceinline__ bool far_scale(int byte) {
    return static_cast<unsigned>(byte - kExpBias + kNearScale) > 2u * kNearScale;
}

// The smallest k with amax <= 448 * 2^k (amax finite, >= 0), within [kExpMin, kExpMax].
// amax = f * 2^e with f in [1, 2), and 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int e = static_cast<int>(bits >> 23) - 127;  // a subnormal or zero gives -127, below kExpMin
    const int k = e - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(k, kExpMin), kExpMax);
}

// Larger of the magnitudes, bf16 pair by pair, as unsigned integers (their order is the
// magnitudes'; infinities and NaN come last).
__device__ __forceinline__ uint32_t max_mag2(uint32_t m, uint32_t w) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w & 0x7fff7fffu));
    return d;
}

// A bf16 pair's magnitudes with infinities and NaN as zero.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    w &= 0x7fff7fffu;
    return ((w & 0xffffu) < 0x7f80u ? w & 0xffffu : 0u) | (w >> 16 < 0x7f80u ? w & 0xffff0000u : 0u);
}

// The four e4m3 codes of a word as f16 pairs: lo the two low bytes, hi the others (exact; a NaN
// code gives NaN).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Bit 7 of every byte says whether that code of the word is a NaN (0x7f and 0xff); the other bits are arbitrary.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }
// 0xff in the bytes that are, 0 in the others.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (nan_bits(w) >> 7 & 0x01010101u) * 0xffu; }

// Four values rounded to nearest even e4m3, lowest byte first (magnitudes past 448 saturate, NaN
// stays NaN).
__device__ __forceinline__ uint32_t to_e4m3x4(float x0, float x1, float x2, float x3) {
    uint32_t d;
    asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\tmov.b32 %0, {a, b};\n\t}"
        : "=r"(d)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return d;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// D[16x8] += A[16x16] * B[16x8], f16 in, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace pa
