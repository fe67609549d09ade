// q8_device.cuh -- what the kernels of the 8-bit cache share: e4m3 conversions,
// operands split into e4m3 parts, the fp8 tensor-core instruction, scales.
#pragma once

#include <cuda_fp16.h>

#include "q8_args.h"
#include "rk_device.cuh"

namespace rk {

// Two floats -> packed e4m3 (lo in the low byte), half to even, saturating.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// The two e4m3 in the low half -> packed FP16, two floats (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    return h;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t w) {
    const uint32_t h = e4m3x2_to_f16x2(w);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
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

// 1 / x, off by at most one unit in the last place.
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Scale exponent of a set of bf16 values from the largest |x| as a bit pattern:
// floor(log2) - 7, at least Q8_E_MIN, so that values over 2^E stay below 2^8
// and their rotation below 362.
__device__ __forceinline__ int q8_exponent(uint32_t amax_bits) { return max((int)(amax_bits >> 7) - 127 - 7, Q8_E_MIN); }

// A scale the attention calls accept: positive, normal, finite.
__device__ __forceinline__ bool scale_ok(float s) { return s >= 1.17549435e-38f && s < INFINITY; }

// Smallest and largest exponent of V's scales that weights of one running maximum have in them.
// Weights have V's scale in their exponent and the sum takes it out again, so a key whose scale is far
// below another's is lost to the sum where its weight passes FP32's 2^-126, which is 2^-133 of the
// largest or less.  With exponents up to 80 apart 2^30 lost keys are 2^-22 of the sum at most; further
// apart the query fails.  One word: the largest exponent, and the largest distance below 255.
struct VSpan {
    uint32_t w = 0;
    __device__ __forceinline__ void add(float scale) {
        const uint32_t e = __float_as_uint(scale) >> 23;
        w = __vmaxu2(w, e << 16 | (255u - e));
    }
    // with the lanes that differ in the bits FROM .. TO / 2 of their number
    template <int FROM, int TO>
    __device__ __forceinline__ void join() {
#pragma unroll
        for (int o = FROM; o < TO; o <<= 1) w = __vmaxu2(w, __shfl_xor_sync(0xffffffffu, w, o));
    }
    __device__ __forceinline__ bool too_wide() const { return (w >> 16) + (w & 0xffffu) > 255u + 80u; }
    // a set that may be too wide with others: not every exponent in [-40, 40]
    __device__ __forceinline__ bool outside() const { return (w >> 16) > 127u + 40u || (w & 0xffffu) > 128u + 40u; }
};

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
// D[tmem] (+)= A[smem] * B[smem], the first kn of 4 k-steps of 32 e4m3 values,
// accumulating from the second on, and at the first iff acc0.  Called by a whole
// converged warp with uniform operands; one elected lane issues.  a_lo, b_lo and
// A_HI, B_HI: descriptor words of the first k-step; A_STEP, B_STEP (16-byte units)
// lead to the next.
template <uint32_t A_STEP, uint32_t B_STEP>
__device__ __forceinline__ void mma_f8_x4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t a_hi, uint32_t b_hi, uint32_t idesc,
                                          uint32_t acc0, int kn) {
    asm volatile(
        "{\n\t.reg .pred p, e, t, k;\n\t.reg .b32 al, bl;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, %6, %6;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t"
        "add.u32 al, %1, %8;\n\tadd.u32 bl, %2, %9;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"
        "setp.gt.and.s32 k, %7, 1, e;\n\t"
        "@k tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, t;\n\t"
        "add.u32 al, al, %8;\n\tadd.u32 bl, bl, %9;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"
        "setp.gt.and.s32 k, %7, 2, e;\n\t"
        "@k tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, t;\n\t"
        "add.u32 al, al, %8;\n\tadd.u32 bl, bl, %9;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"
        "setp.gt.and.s32 k, %7, 3, e;\n\t"
        "@k tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, t;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(acc0), "r"(kn), "n"(A_STEP), "n"(B_STEP)
        : "memory");
}
// High word of an MN-major tile without swizzle: 16 values of a row of K in 16
// bytes, rows 16 bytes apart, so groups of 8 rows (the leading byte offset, in the
// low word) are 128 bytes apart and blocks of 16 columns 2 KiB (128 rows).
constexpr uint32_t DESC_HI_ROWS16 = (2048u >> 4) | (1u << 14);

// By one elected lane of a converged warp, operands uniform: a 5-D box copy, and an
// arrival that expects `bytes` of copies (0: the arrival alone).
__device__ __forceinline__ void tma_load_5d_elect(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2, int c3,
                                                  int c4, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_elect(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                                  uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}
// For what is read once: the first to leave L2.
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void arrive_expect_tx_elect(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes)
        : "memory");
}

// 16-byte asynchronous copy, or 16 zero bytes.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool copy) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16 : 0) : "memory");
}

// 32 lanes x one 32-bit column.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}

}  // namespace rk
