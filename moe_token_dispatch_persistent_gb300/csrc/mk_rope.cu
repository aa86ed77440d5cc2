// mk_rope.cu -- mk_qk_norm_rope: root-mean-square norms of each head of the
// queries and keys, their rotation by position, and the keys' and values' way
// into the pages of a cache, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w                 per head, D columns
//   angle(t, i) = positions[axis(i)][t] * inv_freq[i]   per pair i of columns
//   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Angles.  pos * inv_freq in 32 bits would be off by whole radians for far
// positions.  Of the angle only the part below a turn counts, so a frequency is
// held as the 64-bit fraction of a turn that one position adds, and the angle is
// its product with the position modulo 2^64: exact, three integer products.
//
// A row of D columns is held by D/8 lanes (rounded up to 4, 8, 16 or 32), eight
// columns each; a warp takes one token, or a part of its heads when there are
// few tokens, so that a token's sines are computed once.  Traffic bounds it: 4
// bytes an element and 7 to 10 operations.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mk.h"
#include "mk_fp4.cuh"
#include "mk_host.h"

namespace mk {
namespace {

constexpr int ROPE_MAX_D = 256;
constexpr int ROPE_PAIRS = ROPE_MAX_D / 2;
constexpr int ROPE_AXES = 4;
constexpr int ROPE_WARPS = 8;
constexpr int ROPE_AHEAD = 4;  // rows in flight per lane

struct RopeParams {
    const __nv_bfloat16 *q, *k, *v;
    const __nv_bfloat16 *q_weight, *k_weight;  // or null
    const int32_t* positions;
    const float* inv_freq;
    __nv_bfloat16 *q_out, *k_out, *v_out;      // k_out, v_out or null
    const int64_t* slots;
    uint8_t *k_cache, *v_cache, *k_scales, *v_scales;
    const float *k_factor, *v_factor;          // or null
    DevError* err;
    int64_t q_stride, q_head, k_stride, k_head, v_stride, v_head;
    int64_t position_stride;
    int64_t page_stride, token_stride, head_stride;        // bytes
    int64_t scale_page, scale_token, scale_head;           // bytes
    int64_t capacity;                                      // slots of the pool
    int64_t items;                                         // (token, part of its rows)
    int T, Hq, Hkv, D, rot, page_size, parts;
    int q_steps, k_steps, v_steps;                         // warp's turns over a token's heads
    float eps;
    uint8_t axis[ROPE_PAIRS];
};

// 2^64 times the turns that one position adds: inv_freq / (2 pi), without whole
// turns.  2^64 / (2 pi) has 62 bits, a frequency's significand 24.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
    constexpr uint64_t UNIT = 2935890503282001226ull;  // 2^64 / (2 pi), rounded
    const uint32_t bits = __float_as_uint(fabsf(f));
    const uint32_t e = bits >> 23, m = e ? (bits & 0x7fffffu) | 0x800000u : (bits & 0x7fffffu);
    const int shift = 150 - int(max(e, 1u));  // |f| = m * 2^-shift
    const uint64_t lo = UNIT * m, hi = __umul64hi(UNIT, m);
    uint64_t u;
    if (shift <= 0) u = shift > -64 ? lo << -shift : 0;
    else if (shift < 64) u = (hi << (64 - shift)) | (lo >> shift);
    else u = shift < 128 ? hi >> (shift - 64) : 0;
    return f < 0.f ? 0 - u : u;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}
__device__ __forceinline__ void unpack8(const uint4& q, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = (&q.x)[i];
        y[2 * i] = __uint_as_float(u << 16);
        y[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
    }
}

// LANES hold a row.  HALVES: column i pairs with i + rot/2, else i even with i + 1.
template <int LANES, bool HALVES, int CACHE>
__global__ void __launch_bounds__(ROPE_WARPS * 32) mk_qk_norm_rope_kernel(const RopeParams p) {
    constexpr int ROWS = 32 / LANES;      // rows that a warp holds at a time
    constexpr int MINE = HALVES ? 8 : 4;  // pairs of a lane's columns
    __shared__ __align__(16) float2 table[ROPE_WARPS][ROPE_PAIRS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LANES, l = lane % LANES, c = l * 8;
    const int half = p.rot / 2;
    const bool live = c < p.D, turned = c < p.rot;
    const int pair0 = HALVES ? (c < half ? c : c - half) : c / 2;
    const int partner = HALVES && turned ? (c < half ? lane + half / 8 : lane - half / 8) : lane;
    const int steps = p.q_steps + p.k_steps + p.v_steps;

    uint64_t unit[ROPE_PAIRS / 32];
#pragma unroll
    for (int i = 0; i < ROPE_PAIRS / 32; ++i) {
        const int pair = i * 32 + lane;
        unit[i] = pair < half ? turns_per_position(__ldg(p.inv_freq + pair)) : 0;
    }
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 wq = none, wk = none;
    if (live && p.q_weight) wq = __ldg(reinterpret_cast<const uint4*>(p.q_weight + c));
    if (live && p.k_weight) wk = __ldg(reinterpret_cast<const uint4*>(p.k_weight + c));

    for (int64_t item = int64_t(blockIdx.x) * ROPE_WARPS + warp; item < p.items; item += int64_t(gridDim.x) * ROPE_WARPS) {
        const int t = int(item / p.parts), part = int(item - int64_t(t) * p.parts);
        const int s0 = int(int64_t(steps) * part / p.parts), s1 = int(int64_t(steps) * (part + 1) / p.parts);

        auto load = [&](int s) -> uint4 {
            if (s >= s1 || !live) return none;
            const __nv_bfloat16* row;
            int h = s * ROWS + sub, heads = p.Hq;
            if (s < p.q_steps) {
                row = p.q + t * p.q_stride + h * p.q_head;
            } else if (s < p.q_steps + p.k_steps) {
                h -= p.q_steps * ROWS;
                heads = p.Hkv;
                row = p.k + t * p.k_stride + h * p.k_head;
            } else {
                h -= (p.q_steps + p.k_steps) * ROWS;
                heads = p.Hkv;
                row = p.v + t * p.v_stride + h * p.v_head;
            }
            return h < heads ? *reinterpret_cast<const uint4*>(row + c) : none;
        };
        uint4 x[ROPE_AHEAD];
#pragma unroll
        for (int i = 0; i < ROPE_AHEAD; ++i) x[i] = load(s0 + i);

        // where the token's keys and values go; -1: nowhere
        int64_t page = -1, token = 0;
        if (CACHE != MK_CACHE_NONE) {
            const int64_t slot = __ldg(p.slots + t);
            if (slot >= p.capacity) {
                if (lane == 0) cache_error(p.err, 2u /* fault */, SITE_SLOT_RANGE, uint32_t(t));
            } else if (slot >= 0) {
                page = slot < (int64_t(1) << 31) ? int64_t(uint32_t(slot) / uint32_t(p.page_size)) : slot / p.page_size;
                token = slot - page * p.page_size;
            }
        }

        // sines and cosines of the token's pairs, then of this lane's
        float cs[MINE], sn[MINE];
        if (s0 < p.q_steps + p.k_steps && half > 0) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < ROPE_PAIRS / 32; ++i) {
                const int pair = i * 32 + lane;
                if (pair < half) {
                    const int64_t pos = __ldg(p.positions + p.axis[pair] * p.position_stride + t);
                    const int64_t turn = int64_t(uint64_t(pos) * unit[i]);
                    float sine, cosine;
                    sincospif(float(int32_t(turn >> 32)) * 4.656612873077393e-10f /* 2^-31 */, &sine, &cosine);
                    table[warp][pair] = make_float2(cosine, sine);
                }
            }
            __syncwarp();
            if (turned) {
#pragma unroll
                for (int i = 0; i < MINE; ++i) {
                    const float2 e = table[warp][pair0 + i];
                    cs[i] = e.x;
                    sn[i] = HALVES && c < half ? -e.y : e.y;
                }
            }
        }

        auto norm_and_turn = [&](float (&y)[8], const void* weight, const uint4& w) {
            if (weight) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(y[i], y[i], sum);
#pragma unroll
                for (int d = LANES / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const float rstd = rsqrtf(sum / float(p.D) + p.eps);
                float wf[8];
                unpack8(w, wf);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * wf[i];
            }
            if (HALVES) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, y[i], partner);
                if (turned)
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = fmaf(o[i], sn[i % MINE], y[i] * cs[i % MINE]);
            } else if (turned) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = y[2 * i], b = y[2 * i + 1];
                    y[2 * i] = fmaf(-b, sn[i], a * cs[i]);
                    y[2 * i + 1] = fmaf(a, sn[i], b * cs[i]);
                }
            }
        };
        // a row of keys or values into the cache; `out`: what the cache holds of it, or null
        auto keep = [&](const float (&y)[8], uint8_t* cache, uint8_t* scales, const float* factor, int h, __nv_bfloat16* out) {
            const bool on = live && h < p.Hkv;
            if constexpr (CACHE == MK_CACHE_BF16) {
                const uint4 b = pack8(y);
                if (on && page >= 0)
                    *reinterpret_cast<uint4*>(cache + page * p.page_stride + token * p.token_stride + h * p.head_stride + c * 2) = b;
                if (on && out) *reinterpret_cast<uint4*>(out + c) = b;
            } else if constexpr (CACHE == MK_CACHE_FP4) {
                const float f = factor && on ? __ldg(factor + h) : 1.f;
                float g[8], a = 0.f;
                const Quotient by(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    g[i] = factor ? by.of(y[i]) : y[i];
                    a = max_nan(a, fabsf(g[i]));
                }
                a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
                const uint32_t byte = fp4_scale(a);
                const float scale = float_of_half(halves_of_e4m3x2(byte));
                const Quotient unit_of(scale);
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) w |= e2m1x2_of(unit_of.of(g[2 * i]), unit_of.of(g[2 * i + 1])) << (8 * i);
                if (on && page >= 0) {
                    *reinterpret_cast<uint32_t*>(cache + page * p.page_stride + token * p.token_stride + h * p.head_stride + c / 2) = w;
                    if ((l & 1) == 0)
                        scales[page * p.scale_page + token * p.scale_token + h * p.scale_head + c / FP4_GROUP] = uint8_t(byte);
                }
                if (on && out) {
                    uint32_t e[4];
                    halves_of_e2m1x8(w, e[0], e[1], e[2], e[3]);
                    float held[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        held[2 * i] = float_of_half(e[i]) * scale * f;
                        held[2 * i + 1] = float_of_half(e[i] >> 16) * scale * f;
                    }
                    *reinterpret_cast<uint4*>(out + c) = pack8(held);
                }
            } else {
                if (on && out) *reinterpret_cast<uint4*>(out + c) = pack8(y);
            }
        };

        for (int s = s0; s < s1; s += ROPE_AHEAD) {
#pragma unroll
            for (int i = 0; i < ROPE_AHEAD; ++i) {
                if (s + i >= s1) break;  // the same for the whole warp
                const uint4 raw = x[i];
                float y[8];
                unpack8(raw, y);
                x[i] = load(s + i + ROPE_AHEAD);
                int h = (s + i) * ROWS + sub;
                if (s + i < p.q_steps) {
                    norm_and_turn(y, p.q_weight, wq);
                    if (live && h < p.Hq)
                        *reinterpret_cast<uint4*>(p.q_out + (int64_t(t) * p.Hq + h) * p.D + c) = pack8(y);
                } else if (s + i < p.q_steps + p.k_steps) {
                    h -= p.q_steps * ROWS;
                    norm_and_turn(y, p.k_weight, wk);
                    keep(y, p.k_cache, p.k_scales, p.k_factor, h,
                         p.k_out ? p.k_out + (int64_t(t) * p.Hkv + h) * p.D : nullptr);
                } else {
                    h -= (p.q_steps + p.k_steps) * ROWS;
                    if constexpr (CACHE == MK_CACHE_BF16) {  // as they are
                        if (live && h < p.Hkv && page >= 0)
                            *reinterpret_cast<uint4*>(p.v_cache + page * p.page_stride + token * p.token_stride +
                                                      h * p.head_stride + c * 2) = raw;
                    } else {
                        keep(y, p.v_cache, p.v_scales, p.v_factor, h,
                             p.v_out ? p.v_out + (int64_t(t) * p.Hkv + h) * p.D : nullptr);
                    }
                }
            }
        }
    }
}

template <int LANES, bool HALVES>
void launch_rope(const RopeParams& p, int cache, int grid, cudaStream_t st) {
    if (cache == MK_CACHE_NONE) mk_qk_norm_rope_kernel<LANES, HALVES, MK_CACHE_NONE><<<grid, ROPE_WARPS * 32, 0, st>>>(p);
    else if (cache == MK_CACHE_BF16) mk_qk_norm_rope_kernel<LANES, HALVES, MK_CACHE_BF16><<<grid, ROPE_WARPS * 32, 0, st>>>(p);
    else mk_qk_norm_rope_kernel<LANES, HALVES, MK_CACHE_FP4><<<grid, ROPE_WARPS * 32, 0, st>>>(p);
}
template <int LANES>
void launch_rope(const RopeParams& p, bool halves, int cache, int grid, cudaStream_t st) {
    if (halves) launch_rope<LANES, true>(p, cache, grid, st);
    else launch_rope<LANES, false>(p, cache, grid, st);
}

bool row_strides(const void* base, int64_t token, int64_t head) {
    return host_aligned(base, 16) && token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" mk_status_t mk_qk_norm_rope(const mk_qk_norm_rope_t* a, void* stream) {
    if (!a) return MK_ERR_INVALID_ARG;
    if (a->T < 0 || a->Hq < 1 || a->Hkv < 1 || a->D < 16 || a->D % 16 != 0 || a->rot < 0 || a->rot % 16 != 0 || a->rot > a->D)
        return MK_ERR_INVALID_ARG;
    if (a->axes < 1 || a->pairs < MK_PAIR_HALVES || a->pairs > MK_PAIR_NEIGHBOURS || a->cache < MK_CACHE_NONE ||
        a->cache > MK_CACHE_FP4 || a->reserved != 0)
        return MK_ERR_INVALID_ARG;
    if (a->D > ROPE_MAX_D || a->axes > ROPE_AXES || a->Hq > 65536 || a->Hkv > 65536) return MK_ERR_UNSUPPORTED;
    if (!(a->eps >= 0.f) || std::isinf(a->eps)) return MK_ERR_INVALID_ARG;
    const bool stored = a->cache != MK_CACHE_NONE, fp4 = a->cache == MK_CACHE_FP4;
    if (stored && (a->page_size < 1 || a->num_pages < 0)) return MK_ERR_INVALID_ARG;
    if (a->axes > 1 && a->rot > 0 && !a->pair_axis) return MK_ERR_INVALID_ARG;
    if (a->pair_axis)
        for (int i = 0; i < a->rot / 2; ++i)
            if (a->pair_axis[i] >= a->axes) return MK_ERR_INVALID_ARG;
    if (a->T > 0) {
        if (!a->q || !a->k || !a->q_out || (!stored && !a->k_out) || (!fp4 && a->v_out)) return MK_ERR_INVALID_ARG;
        // the stride of a dimension of one is never used
        const auto used = [](int n, int64_t s) { return n > 1 ? s : int64_t(0); };
        if (!row_strides(a->q, used(a->T, a->q_stride), used(a->Hq, a->q_head_stride)) ||
            !row_strides(a->k, used(a->T, a->k_stride), used(a->Hkv, a->k_head_stride)))
            return MK_ERR_INVALID_ARG;
        if (!host_aligned(a->q_out, 16) || !host_aligned(a->k_out, 16) || !host_aligned(a->v_out, 16) ||
            !host_aligned(a->q_weight, 16) || !host_aligned(a->k_weight, 16))
            return MK_ERR_INVALID_ARG;
        if (a->rot > 0 && (!a->positions || !a->inv_freq || !host_aligned(a->positions, 4) || !host_aligned(a->inv_freq, 4)))
            return MK_ERR_INVALID_ARG;
        if (stored) {
            if (!a->v || !a->slots || !host_aligned(a->slots, 8) ||
                !row_strides(a->v, used(a->T, a->v_stride), used(a->Hkv, a->v_head_stride)))
                return MK_ERR_INVALID_ARG;
            if (a->num_pages > 0 && (!a->k_cache || !a->v_cache || (fp4 && (!a->k_scales || !a->v_scales))))
                return MK_ERR_INVALID_ARG;
            const size_t align = fp4 ? 4 : 16;
            const int64_t unit = fp4 ? 4 : 8;
            if (!host_aligned(a->k_cache, align) || !host_aligned(a->v_cache, align)) return MK_ERR_INVALID_ARG;
            for (const int64_t v : {used(a->num_pages, a->page_stride), used(a->page_size, a->token_stride), used(a->Hkv, a->head_stride)})
                if (v < 0 || v % unit != 0) return MK_ERR_INVALID_ARG;
            if (fp4)
                for (const int64_t v : {used(a->num_pages, a->scale_page_stride), used(a->page_size, a->scale_token_stride),
                                        used(a->Hkv, a->scale_head_stride)})
                    if (v < 0) return MK_ERR_INVALID_ARG;
            if (!host_aligned(a->k_factor, 4) || !host_aligned(a->v_factor, 4)) return MK_ERR_INVALID_ARG;
        }
    }
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    const mk_status_t s = host_device(&dev, &sms, &err);
    if (s != MK_OK) return s;
    if (a->T == 0) return MK_OK;

    RopeParams p{};
    p.q = static_cast<const __nv_bfloat16*>(a->q);
    p.k = static_cast<const __nv_bfloat16*>(a->k);
    p.v = static_cast<const __nv_bfloat16*>(a->v);
    p.q_weight = static_cast<const __nv_bfloat16*>(a->q_weight);
    p.k_weight = static_cast<const __nv_bfloat16*>(a->k_weight);
    p.positions = a->positions;
    p.inv_freq = a->inv_freq;
    p.q_out = static_cast<__nv_bfloat16*>(a->q_out);
    p.k_out = static_cast<__nv_bfloat16*>(a->k_out);
    p.v_out = static_cast<__nv_bfloat16*>(a->v_out);
    p.slots = a->slots;
    p.k_cache = static_cast<uint8_t*>(a->k_cache);
    p.v_cache = static_cast<uint8_t*>(a->v_cache);
    p.k_scales = static_cast<uint8_t*>(a->k_scales);
    p.v_scales = static_cast<uint8_t*>(a->v_scales);
    p.k_factor = fp4 ? a->k_factor : nullptr;
    p.v_factor = fp4 ? a->v_factor : nullptr;
    p.err = err;
    p.q_stride = a->q_stride;
    p.q_head = a->q_head_stride;
    p.k_stride = a->k_stride;
    p.k_head = a->k_head_stride;
    p.v_stride = a->v_stride;
    p.v_head = a->v_head_stride;
    p.position_stride = a->position_stride;
    const int64_t size = fp4 ? 1 : 2;
    p.page_stride = a->page_stride * size;
    p.token_stride = a->token_stride * size;
    p.head_stride = a->head_stride * size;
    p.scale_page = a->scale_page_stride;
    p.scale_token = a->scale_token_stride;
    p.scale_head = a->scale_head_stride;
    p.capacity = stored ? int64_t(a->num_pages) * a->page_size : 0;
    p.T = a->T;
    p.Hq = a->Hq;
    p.Hkv = a->Hkv;
    p.D = a->D;
    p.rot = a->rot;
    p.page_size = std::max(1, a->page_size);
    p.eps = a->eps;
    if (a->pair_axis) std::copy(a->pair_axis, a->pair_axis + a->rot / 2, p.axis);
    const int lanes = a->D <= 32 ? 4 : a->D <= 64 ? 8 : a->D <= 128 ? 16 : 32, rows = 32 / lanes;
    p.q_steps = (a->Hq + rows - 1) / rows;
    p.k_steps = (a->Hkv + rows - 1) / rows;
    p.v_steps = stored ? p.k_steps : 0;
    const int steps = p.q_steps + p.k_steps + p.v_steps;
    // A warp per token when the tokens alone fill the GPU twice over, else as many
    // parts of a token's heads as fill it.
    const int64_t room = int64_t(sms) * ROPE_WARPS * 8;
    p.parts = int(std::max<int64_t>(1, std::min<int64_t>(steps, room / a->T)));
    p.items = int64_t(a->T) * p.parts;
    const int grid = int(std::min<int64_t>((p.items + ROPE_WARPS - 1) / ROPE_WARPS, int64_t(sms) * 8));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool halves = a->pairs == MK_PAIR_HALVES;
    if (lanes == 4) launch_rope<4>(p, halves, a->cache, grid, st);
    else if (lanes == 8) launch_rope<8>(p, halves, a->cache, grid, st);
    else if (lanes == 16) launch_rope<16>(p, halves, a->cache, grid, st);
    else launch_rope<32>(p, halves, a->cache, grid, st);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
