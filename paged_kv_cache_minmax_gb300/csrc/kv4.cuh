// kv4.cuh -- the 4-bit cache's number format and page layout (device helpers).
//
// A held value is an e2m1 code times the e4m3 scale of its 16 channels (times
// a factor of the call).  The product of the two has at most 2 + 4 significant
// bits, a magnitude of at most 6 * 448 and no bit below 2^-10 (0.5 * 2^-9), so
// it is exact in fp16 and in bf16.
#pragma once

#include "common.cuh"

namespace kvmm {

// Byte offsets inside a page of T tokens: key codes [T][D/2], key scales
// [T][D/16], then the values' codes and scales the same way.
template <int D, int T>
struct Kv4Page {
    static constexpr int kRow = D / 2;     // codes of one token
    static constexpr int kGroups = D / 16; // scales of one token
    static constexpr int kKeyScales = T * kRow;
    static constexpr int kValues = kKeyScales + T * kGroups;
    static constexpr int kValueScales = kValues + T * kRow;
    static constexpr int kBytes = kValueScales + T * kGroups;
    static_assert(kBytes % 16 == 0 && kValues % 16 == 0, "a page is copied in 16-byte pieces");
};

// shared-memory loads at a 32-bit address plus a constant
template <int OFF>
__device__ __forceinline__ uint4 lds_v4(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a), "n"(OFF));
    return v;
}
template <int OFF>
__device__ __forceinline__ uint2 lds_v2(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(OFF));
    return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_u32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(OFF));
    return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_u16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v) : "r"(a), "n"(OFF));
    return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_u8(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=r"(v) : "r"(a), "n"(OFF));
    return v;
}

__device__ __forceinline__ void sts_u32(uint32_t a, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// mbar_arrive_expect_tx and bulk_copy_g2s_hint at 32-bit shared-memory addresses
__device__ __forceinline__ void mbar_arrive_expect_tx_at(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy_g2s_hint_at(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                                      uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
        "%4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// byte i of w as two e2m1 codes -> two halves (low nibble in the low half), exact
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_half2(uint32_t w)
{
    uint32_t d;
    if (I == 0)
        asm("{.reg .b8 a, b, c, e; mov.b32 {a, b, c, e}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(d) : "r"(w));
    else if (I == 1)
        asm("{.reg .b8 a, b, c, e; mov.b32 {a, b, c, e}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(d) : "r"(w));
    else if (I == 2)
        asm("{.reg .b8 a, b, c, e; mov.b32 {a, b, c, e}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(d) : "r"(w));
    else
        asm("{.reg .b8 a, b, c, e; mov.b32 {a, b, c, e}, %1; cvt.rn.f16x2.e2m1x2 %0, e;}" : "=r"(d) : "r"(w));
    return d;
}

// the two low bytes of w as e4m3 -> two halves, exact
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t w)
{
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(w)));
    return d;
}

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float half_lo(uint32_t w)
{
    float f;
    asm("{.reg .f16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l;}" : "=f"(f) : "r"(w));
    return f;
}
__device__ __forceinline__ float half_hi(uint32_t w)
{
    float f;
    asm("{.reg .f16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, h;}" : "=f"(f) : "r"(w));
    return f;
}

// round two floats to fp16 (nearest even) and pack: lo in bits 0..15
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// nearest e4m3 of x >= 0 (ties to even, at most 448)
__device__ __forceinline__ uint32_t float_to_e4m3(float x)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(x));
    return d;
}

// nearest e2m1 of two floats (ties to even, at most 6 in magnitude): lo in the low nibble
__device__ __forceinline__ uint32_t float2_to_e2m1x2(float lo, float hi)
{
    uint32_t d;
    asm("{.reg .b8 t, z; mov.b16 {t, z}, 0; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; mov.b32 %0, {t, z, z, z};}"
        : "=r"(d)
        : "f"(hi), "f"(lo));
    return d;
}

// D(16x8, f32) += A(16x16, f16, row) * B(16x8, f16, col), fragments as mma_bf16_16816
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace kvmm
