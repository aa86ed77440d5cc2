// mk_quant.cuh -- the 8-bit format that the norm writes and the expert layer
// reads and keeps h in: e4m3 values with a scale per row and 128 columns,
// a = max |y|, scale = a / 448 (1 where a < 2^-100), value = e4m3(y / scale).
#pragma once

#include <cuda_runtime.h>

#include <cmath>

namespace mk {

constexpr float E4M3_MAX = 448.f;
constexpr float TINY_GROUP = 7.888609052210118e-31f;  // 2^-100

// The larger of the two, NaN if either is (fmaxf would drop it, and with it a
// row that holds NaN would get a finite scale).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Division by a group's scale: the product with its reciprocal, corrected once
// by what it leaves of y (Markstein 1990).  The product alone is off by up to
// an ulp and a half, which takes values next to the middle of two e4m3 values
// to the wrong one; a division per value instead costs the norm 10% (97 to 108
// us on 16384 x 4096), the correction 1%.
struct GroupScale {
    float scale, inv, rest;

    __device__ __forceinline__ explicit GroupScale(float a) {
        scale = a < TINY_GROUP ? 1.f : a / E4M3_MAX;
        inv = 1.f / scale;
        rest = scale == INFINITY ? 0.f : scale;  // by infinity: 0, not what 0 * infinity leaves
    }
    __device__ __forceinline__ float of(float y) const {
        const float q = y * inv;
        return fmaf(fmaf(-q, rest, y), inv, q);
    }
};

}  // namespace mk
