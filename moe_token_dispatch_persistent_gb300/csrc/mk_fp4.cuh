// mk_fp4.cuh -- the 4-bit format of a key-value cache: e2m1 values (0, 0.5, 1,
// 1.5, 2, 3, 4, 6 and a sign), two to a byte with the even column in the low
// half, and an e4m3 scale per row of 16 columns.  Of y, divided by its head's
// factor: scale = e4m3(max |y| / 6), at least 2^-9; value = e2m1(y / scale).
// value * scale has 6 significant bits at most, so it is exact in fp16.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mk_host.h"
#include "mk_quant.cuh"

namespace mk {

constexpr int FP4_GROUP = 16;  // columns per scale

// Sites of device errors of the cache's operators (mk_last_error_detail()),
// after those of mk_common.h.
enum CacheSite : int {
    SITE_SLOT_RANGE = 23,    // a slot outside the pool; info: the token
    SITE_SEQUENCE = 24,      // a sequence outside the table, or named twice; info: its place in the list
    SITE_POOL_FULL = 25,     // too few free pages, or too few entries in a row of the table; info: those missing, 2^31 - 1 at most
    SITE_PAGE_INDEX = 26,    // a page outside the pool; info: the page
    SITE_TOKEN_COUNT = 27,   // a count of new tokens outside [0, most], or a length below 0; info: its place in the list
};

__device__ __forceinline__ void cache_error(DevError* e, uint32_t code, uint32_t site, uint32_t info) {
    if (atomicCAS(&e->code, 0u, code) == 0u) {
        e->site = site;
        e->cta = blockIdx.x;
        e->info = info;
    }
}

// e4m3 byte of a value that is not negative; NaN gives 0x7f.
__device__ __forceinline__ uint32_t e4m3_of(float a) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(a));
    return r & 0xffu;
}
// Two e4m3 bytes as two fp16 values, the low byte in the low half.
__device__ __forceinline__ uint32_t halves_of_e4m3x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
    return r;
}
__device__ __forceinline__ float float_of_half(uint32_t h) {
    float r;
    asm("cvt.f32.f16 %0, %1;" : "=f"(r) : "h"(uint16_t(h)));
    return r;
}
// Two values as a byte of e2m1, `lo` in the low half; beyond 6 they are 6.
__device__ __forceinline__ uint32_t e2m1x2_of(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
// The four bytes of a word of e2m1 as four pairs of fp16 values.
__device__ __forceinline__ void halves_of_e2m1x8(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
        : "r"(w));
}

// Packed pairs of fp32.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, r;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 r, a, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// y / f of finite y as the division would round it: the product with the
// reciprocal, corrected once by what it leaves of y (see GroupScale).
struct Quotient {
    float f, inv;

    __device__ __forceinline__ explicit Quotient(float by) : f(by), inv(1.f / by) {}
    __device__ __forceinline__ float of(float y) const {
        const float q = y * inv;
        return fmaf(fmaf(-q, f, y), inv, q);
    }
    __device__ __forceinline__ float2 of(float2 y) const {
        const float2 i2 = make_float2(inv, inv), q = mul2(y, i2);
        return fma2(fma2(q, make_float2(-f, -f), y), i2, q);
    }
};

// Scale of a group whose largest magnitude is a: its byte, at least 1 (2^-9,
// the smallest e4m3 value above 0).
__device__ __forceinline__ uint32_t fp4_scale(float a) { return max(e4m3_of(a / 6.f), 1u); }

}  // namespace mk
