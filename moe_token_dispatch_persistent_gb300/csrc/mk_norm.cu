// mk_norm.cu -- mk_add_rmsnorm: the residual's addition, the root-mean-square
// norm, and its output in bf16 and / or e4m3 with a scale per 128 columns.
//
//   z = x + residual                      residual_out = bf16(z)
//   y = z * rsqrt(mean(z^2) + eps) * w    out = bf16(y)
//   per row and 128 columns: a = max |y|, scale = a / 448 (1 where a < 2^-100),
//   out8 = e4m3(y / scale)
//
// z and y stay in 32-bit registers: the norm and the 8-bit values come from
// the unrounded sum, and each output is rounded once.  One pass: a row is
// read once, held by the warps that share it, and every output is written
// from those registers.  Traffic bounds it (up to 9 bytes an element for 6
// operations); for a few rows the latency of one launch does.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mk.h"
#include "mk_host.h"
#include "mk_quant.cuh"

namespace mk {
namespace {

constexpr int NORM_CHUNK = 256;  // columns of a row that one warp takes at a time: 8 per lane, two 8-bit groups
constexpr int NORM_GROUP = 128;  // columns per scale
constexpr int NORM_MAX_H = 32768;
constexpr int NORM_MAX_WARPS = 32;

struct NormParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* residual;  // or null
    const __nv_bfloat16* weight;
    __nv_bfloat16* out;             // or null
    __nv_bfloat16* residual_out;    // or null
    uint8_t* out8;                  // or null
    float* scale;
    int64_t x_stride, residual_stride;  // elements between rows
    int T, H;
    int warps_per_row, rows_per_cta;
    float eps;
};

// Column of element i of a lane's eight in a chunk.  VEC: eight neighbours
// (16-byte accesses), so lanes 0-15 hold the chunk's first group of 128 and
// lanes 16-31 its second.  Otherwise 32 apart, so elements 0-3 of all lanes
// are the first group and 4-7 the second, and accesses still coalesce.
template <bool VEC>
__device__ __forceinline__ int column(int chunk, int lane, int i) {
    return chunk * NORM_CHUNK + (VEC ? lane * 8 + i : lane + 32 * i);
}

// A lane's eight elements of a chunk, two to a word, zeros past the row's end.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* row, int chunk, int lane, int H) {
    if constexpr (VEC) {
        const int c = column<true>(chunk, lane, 0);
        return c < H ? __ldcs(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t u[4];
        const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c0 = column<false>(chunk, lane, 2 * i), c1 = column<false>(chunk, lane, 2 * i + 1);
            u[i] = (c0 < H ? uint32_t(r[c0]) : 0u) | (c1 < H ? uint32_t(r[c1]) << 16 : 0u);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
}

__device__ __forceinline__ float element(const uint4& q, int i) {
    const uint32_t u = (&q.x)[i >> 1];
    return __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int chunk, int lane, int H, const float (&v)[8]) {
    if constexpr (VEC) {
        const int c = column<true>(chunk, lane, 0);
        if (c >= H) return;
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        __stcs(reinterpret_cast<uint4*>(row + c), make_uint4(u[0], u[1], u[2], u[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = column<false>(chunk, lane, i);
            if (c < H) row[c] = __float2bfloat16_rn(v[i]);
        }
    }
}

// The chunk's two groups in e4m3 with their scales.
template <bool VEC>
__device__ __forceinline__ void quantize8(uint8_t* row, float* scale_row, int chunk, int lane, int H,
                                          const float (&y)[8]) {
    float a[2];
    if constexpr (VEC) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(y[i]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        a[0] = a[1] = m;  // of this lane's own half: one of the two groups
    } else {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max_nan(m, fabsf(y[4 * g + i]));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
            a[g] = m;
        }
    }
    const GroupScale s[2] = {GroupScale(a[0]), GroupScale(a[1])};
    const int group = chunk * 2 + (VEC ? lane >> 4 : lane & 1);
    if (VEC ? (lane & 15) == 0 : lane < 2)
        if (group * NORM_GROUP < H) scale_row[group] = (!VEC && (lane & 1)) ? s[1].scale : s[0].scale;
    uint32_t q[4];  // two values each
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const GroupScale& g = s[VEC ? 0 : i >> 1];
        q[i] = __nv_cvt_float2_to_fp8x2(make_float2(g.of(y[2 * i]), g.of(y[2 * i + 1])), __NV_SATFINITE, __NV_E4M3);
    }
    if constexpr (VEC) {
        const int c = column<true>(chunk, lane, 0);
        if (c < H) __stcs(reinterpret_cast<uint2*>(row + c), make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = column<false>(chunk, lane, i);
            if (c < H) row[c] = uint8_t(q[i >> 1] >> (8 * (i & 1)));
        }
    }
}

// C chunks of a row per warp; warps_per_row * C chunks cover the row, and a
// CTA's rows_per_cta rows are reduced together.  CTAs stay and take further
// rows, whose loads are issued before the current ones are worked on (a CTA
// per row instead: 107 us, not 97, for 16384 x 4096 with every output, 6.2
// TB/s); the weights are loaded once.
template <bool VEC, int C>
__global__ void __launch_bounds__(NORM_MAX_WARPS * 32) mk_add_rmsnorm_kernel(const NormParams p) {
    __shared__ float part[2][NORM_MAX_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wpr = p.warps_per_row;
    const int mine = warp % wpr, first = warp - mine;
    const int H = p.H, groups = (H + NORM_GROUP - 1) / NORM_GROUP;
    const int64_t stride = int64_t(gridDim.x) * p.rows_per_cta;
    // Whether a thread has registers for the next row and the weights.  If not, a
    // row is loaded in its own turn and the weights come from L1 (with them in registers
    // and spills for it: 2048 x 32768 154 us, so 108; 8192 x 7167 242, so 144; 2048 x
    // 32767 650, so 300).  At 64 registers 20 bytes are spilled with VEC and two chunks,
    // 100 without VEC and four; the other forms have none.
    constexpr bool AHEAD = C <= (VEC ? 2 : 1);
    uint4 x[C], r[C], w[C];
    auto fetch = [&](int64_t row) {
        if (row >= p.T) return;
#pragma unroll
        for (int j = 0; j < C; ++j) x[j] = load8<VEC>(p.x + row * p.x_stride, mine + j * wpr, lane, H);
        if (p.residual)
#pragma unroll
            for (int j = 0; j < C; ++j) r[j] = load8<VEC>(p.residual + row * p.residual_stride, mine + j * wpr, lane, H);
    };
    int64_t base = int64_t(blockIdx.x) * p.rows_per_cta;
    if (AHEAD) {
        fetch(base + warp / wpr);
#pragma unroll
        for (int j = 0; j < C; ++j) w[j] = load8<VEC>(p.weight, mine + j * wpr, lane, H);
    }
    for (int turn = 0; base < p.T; base += stride, turn ^= 1) {
        const int64_t row = base + warp / wpr;
        const bool live = row < p.T;
        float z[C][8];
        float sum = 0.f;
        if (live) {
            if (!AHEAD) fetch(row);
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    z[j][i] = element(x[j], i);
                    if (p.residual) z[j][i] += element(r[j], i);
                    sum = fmaf(z[j][i], z[j][i], sum);
                }
            if (AHEAD) fetch(row + stride);
            if (p.residual_out)
#pragma unroll
                for (int j = 0; j < C; ++j) store8<VEC>(p.residual_out + row * H, mine + j * wpr, lane, H, z[j]);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (wpr > 1) {  // the same for the whole CTA
            if (lane == 0) part[turn][warp] = sum;
            __syncthreads();
            sum = lane < wpr ? part[turn][first + lane] : 0.f;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        }
        if (!live) continue;
        const float rstd = rsqrtf(sum / float(H) + p.eps);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (!AHEAD) w[j] = load8<VEC>(p.weight, mine + j * wpr, lane, H);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] = z[j][i] * rstd * element(w[j], i);
            if (p.out) store8<VEC>(p.out + row * H, mine + j * wpr, lane, H, z[j]);
            if (p.out8) quantize8<VEC>(p.out8 + row * H, p.scale + row * groups, mine + j * wpr, lane, H, z[j]);
        }
    }
}

template <bool VEC>
void launch_norm(const NormParams& p, int per_warp, int grid, cudaStream_t st) {
    const int threads = p.warps_per_row * p.rows_per_cta * 32;
    if (per_warp == 1) mk_add_rmsnorm_kernel<VEC, 1><<<grid, threads, 0, st>>>(p);
    else if (per_warp == 2) mk_add_rmsnorm_kernel<VEC, 2><<<grid, threads, 0, st>>>(p);
    else mk_add_rmsnorm_kernel<VEC, 4><<<grid, threads, 0, st>>>(p);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" mk_status_t mk_add_rmsnorm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                      const void* weight, int T, int H, float eps, void* out, void* out8, float* scale,
                                      void* residual_out, void* stream) {
    if (T < 0 || H < 1) return MK_ERR_INVALID_ARG;
    if (H > NORM_MAX_H) return MK_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || std::isinf(eps)) return MK_ERR_INVALID_ARG;
    if (T > 0) {
        if (!x || !weight || (!out && !out8) || (out8 != nullptr) != (scale != nullptr)) return MK_ERR_INVALID_ARG;
        if (residual_out && !residual) return MK_ERR_INVALID_ARG;
        if (!host_aligned(x, 2) || !host_aligned(residual, 2) || !host_aligned(weight, 2) || !host_aligned(out, 2) ||
            !host_aligned(residual_out, 2) || !host_aligned(scale, 4))
            return MK_ERR_INVALID_ARG;
        if (T > 1 && (x_stride < H || (residual && residual_stride < H))) return MK_ERR_INVALID_ARG;
    }
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    const mk_status_t s = host_device(&dev, &sms, &err);
    if (s != MK_OK) return s;
    if (T == 0) return MK_OK;

    NormParams p{};
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.residual = static_cast<const __nv_bfloat16*>(residual);
    p.weight = static_cast<const __nv_bfloat16*>(weight);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.residual_out = static_cast<__nv_bfloat16*>(residual_out);
    p.out8 = static_cast<uint8_t*>(out8);
    p.scale = scale;
    p.x_stride = x_stride;
    p.residual_stride = residual_stride;
    p.T = T;
    p.H = H;
    p.eps = eps;
    const bool vec = H % 8 == 0 && (T == 1 || (x_stride % 8 == 0 && (!residual || residual_stride % 8 == 0))) &&
                     host_aligned(x, 16) && host_aligned(residual, 16) && host_aligned(weight, 16) &&
                     host_aligned(out, 16) && host_aligned(residual_out, 16) && host_aligned(out8, 8);
    const int chunks = (H + NORM_CHUNK - 1) / NORM_CHUNK;
    // A chunk per warp while two CTAs fit an SM (16 warps a row), or as far as a
    // CTA's 32 warps go when there is no more than a row per SM (all of a row is
    // then loaded at once); two or four beyond.  8192 x 7168: 85 us with two
    // chunks per warp, 92 with one.
    const bool one = chunks <= NORM_MAX_WARPS / 2 || (T <= sms && chunks <= NORM_MAX_WARPS);
    const int per_warp = one ? 1 : chunks <= 2 * NORM_MAX_WARPS ? 2 : 4;
    p.warps_per_row = (chunks + per_warp - 1) / per_warp;
    p.rows_per_cta = p.warps_per_row >= 8 ? 1 : 8 / p.warps_per_row;
    const int64_t wanted = (int64_t(T) + p.rows_per_cta - 1) / p.rows_per_cta;
    const int resident = std::max(1, 1024 / (p.warps_per_row * p.rows_per_cta * 32));  // at 64 registers a thread
    const int grid = int(std::min<int64_t>(wanted, int64_t(sms) * resident));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (vec) launch_norm<true>(p, per_warp, grid, st);
    else launch_norm<false>(p, per_warp, grid, st);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
