// q8_device.cuh -- what the kernels of the 8-bit cache share: e4m3 conversions,
// operands split into e4m3 parts, the fp8 tensor-core instruction, scales.
#pragma once

#include <cuda_fp16.h>

#include "rk_device.cuh"

namespace rk {

// Two floats -> packed e4m3 (lo in the low byte), half to even, saturating.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Packed e4m3 -> two floats (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// x (two values) as a sum of e4m3 parts: the part, and x reduced to what is left
// (exact in FP32).  A part keeps 4 significant bits, so it leaves at most 2^-4
// of the value, or 2^-10 where that is less than e4m3's smallest step.
__device__ __forceinline__ uint32_t take_part(float2& x) {
    const uint32_t p = cvt_e4m3x2(x.x, x.y);
    const float2 f = e4m3x2_to_float2(p);
    x.x -= f.x;
    x.y -= f.y;
    return p;
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Scale exponent of a set of bf16 values from the largest |x| as a bit pattern:
// floor(log2) - 7, at least Q8_E_MIN, so that values over 2^E stay below 2^8
// and their rotation below 362.
__device__ __forceinline__ int q8_exponent(uint32_t amax_bits) { return max((int)(amax_bits >> 7) - 127 - 7, Q8_E_MIN); }

// A scale the attention calls accept: positive, normal, finite.
__device__ __forceinline__ bool scale_ok(float s) { return s >= 1.17549435e-38f && s < INFINITY; }

// Largest of a warp's values (NaN left out), in every lane.
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Instruction descriptor of kind::f8f6f4, e4m3 A and B, FP32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N, int a_mn_major, int b_mn_major) {
    return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[smem] * B[smem], k-steps KS .. END - 1 of 32 e4m3 values,
// accumulating from k-step 1 on, and at k-step 0 iff acc0.  Called by a whole
// converged warp with uniform operands; one elected lane issues.  a_lo, b_lo:
// descriptor low words of k-step 0, A_STEP / B_STEP added for each (16-byte units,
// immediates, so that a step costs the issuing warp no arithmetic).  A lies in a
// 128-byte-swizzled tile (high word DESC_HI), B in one with high word B_HI.
template <int KS, int END, uint32_t A_STEP, uint32_t B_STEP, uint32_t B_HI>
__device__ __forceinline__ void mma_f8_steps(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc0) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 al, bl;\n\t.reg .b64 da, db;\n\t"
        "add.u32 al, %1, %5;\n\tadd.u32 bl, %2, %6;\n\t"
        "mov.b64 da, {al, %4};\n\tmov.b64 db, {bl, %8};\n\t"
        "setp.ne.b32 p, %7, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(DESC_HI), "n"(KS * A_STEP), "n"(KS * B_STEP), "r"(KS > 0 ? 1u : acc0), "r"(B_HI)
        : "memory");
    if constexpr (KS + 1 < END) mma_f8_steps<KS + 1, END, A_STEP, B_STEP, B_HI>(d, a_lo, b_lo, idesc, acc0);
}
// High word of an MN-major tile without swizzle: 16 values of a row of K in 16
// bytes, rows 16 bytes apart, so groups of 8 rows (the leading byte offset, in the
// low word) are 128 bytes apart and blocks of 16 columns 2 KiB (128 rows).
constexpr uint32_t DESC_HI_ROWS16 = (2048u >> 4) | (1u << 14);

// 32 lanes x one 32-bit column.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}

}  // namespace rk
