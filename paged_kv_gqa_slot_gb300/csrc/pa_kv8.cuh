// pa_kv8.cuh -- the 8-bit pool's number format on the device, shared by the kernels that
// write it (pa_append8.cu) and read it (pa_decode8.cu, the prefill kernels).
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

// The smallest k with amax <= 448 * 2^k (amax finite, >= 0), within [kExpMin, kExpMax].
// amax = f * 2^e with f in [1, 2), and 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int e = static_cast<int>(bits >> 23) - 127;  // a subnormal or zero gives -127, below kExpMin
    const int k = e - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(k, kExpMin), kExpMax);
}

// Two e4m3 codes as f16 (exact; a NaN code gives NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair16) {
    uint32_t d;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(pair16));
    return d;
}

// lo and hi rounded to nearest even e4m3 (magnitudes past 448 saturate, NaN stays NaN).
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint32_t d;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(d)
        : "f"(lo), "f"(hi));
    return d;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The four codes of a word times `s` as four bf16 (two packed words).  With s = 2^k of an
// 8-bit pool the products are bf16 numbers, so nothing is rounded.
__device__ __forceinline__ uint2 e4m3x4_to_bf16x4(uint32_t w, float s) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(w & 0xffffu));
    const float2 b = f16x2_to_float2(e4m3x2_to_f16x2(w >> 16));
    return make_uint2(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s));
}

// D[16x8] += A[16x16] * B[16x8], f16 in, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Asynchronous copies of 16 (around L1) or 8 bytes into shared memory, completion in groups
// that the issuing thread commits and waits for.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace pa
