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
// its product with the position modulo 2^64: exact, three integer products.  Its
// distance from the nearest quarter turn is what the functions get.
//
// A row of D columns is held by D/8 lanes (rounded up to 4, 8, 16 or 32), eight
// columns each, four whole pairs; a warp takes one token, or a part of its heads
// when there are few tokens, so that a token's sines are computed once.  Traffic
// bounds it, 4 bytes an element for 7 to 10 operations, but not by far: 16384
// tokens of 32 + 2 * 8 heads of 128 into bf16 pages take 70 us (5.8 TB/s, 96
// instructions for two rows; with partner columns in other lanes 184, 126 us),
// 8192 of them into 4-bit pages 51 us; one token 3.5 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

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
constexpr int ROPE_CTAS = 4;   // of an SM: 64 registers a thread (some forms spill for it, up to 44 words)

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

// A lane's four pairs (a, b) of columns, the first two and the last two pairs side
// by side.  HALVES: a's are four neighbouring columns, in x and y, and b's another
// four, in z and w; else a's are the low halves of the four words.
struct Pairs {
    float2 a[2], b[2];
};
template <bool HALVES>
__device__ __forceinline__ Pairs unpack_pairs(const uint4& q) {
    const auto lo = [](uint32_t u) { return __uint_as_float(u << 16); };
    const auto hi = [](uint32_t u) { return __uint_as_float(u & 0xffff0000u); };
    Pairs p;
    if constexpr (HALVES) {
        p.a[0] = make_float2(lo(q.x), hi(q.x));
        p.a[1] = make_float2(lo(q.y), hi(q.y));
        p.b[0] = make_float2(lo(q.z), hi(q.z));
        p.b[1] = make_float2(lo(q.w), hi(q.w));
    } else {
        p.a[0] = make_float2(lo(q.x), lo(q.y));
        p.b[0] = make_float2(hi(q.x), hi(q.y));
        p.a[1] = make_float2(lo(q.z), lo(q.w));
        p.b[1] = make_float2(hi(q.z), hi(q.w));
    }
    return p;
}
template <bool HALVES>
__device__ __forceinline__ uint4 pack_pairs(const Pairs& p) {
    if constexpr (HALVES)
        return make_uint4(pack2(p.a[0].x, p.a[0].y), pack2(p.a[1].x, p.a[1].y), pack2(p.b[0].x, p.b[0].y), pack2(p.b[1].x, p.b[1].y));
    else
        return make_uint4(pack2(p.a[0].x, p.b[0].x), pack2(p.a[0].y, p.b[0].y), pack2(p.a[1].x, p.b[1].x), pack2(p.a[1].y, p.b[1].y));
}

// LANES hold a row, eight columns each.  HALVES: column i pairs with i + rot/2, else
// i even with i + 1.  A lane's columns are four pairs, so a rotation stays in it:
// with HALVES 4l .. and rot/2 + 4l .., otherwise, and past rot, 8l ..
// WHOLE: every lane has columns, and all of them are rotated.
template <int LANES, bool HALVES, int CACHE, bool WHOLE>
__global__ void __launch_bounds__(ROPE_WARPS * 32, ROPE_CTAS) mk_qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int ROWS = 32 / LANES;  // rows that a warp holds at a time
    // 4-bit keys with HALVES: a scale's 16 columns lie in two neighbouring lanes only if a
    // lane's eight follow one another, so the two of a pair meet by a shuffle.
    constexpr bool KEYS_IN_ORDER = HALVES && CACHE == MK_CACHE_FP4;
    constexpr int PAIRS = LANES * 4;
    __shared__ uint64_t units[PAIRS];
    __shared__ __align__(16) float2 table[ROPE_WARPS][PAIRS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LANES, l = lane % LANES, c = l * 8;
    const int D = WHOLE ? LANES * 8 : p.D, rot = WHOLE ? D : p.rot, half = rot / 2;
    const bool live = WHOLE || c < D, turned = WHOLE || c < rot;
    const int c0 = HALVES && turned ? l * 4 : c, c1 = HALVES && turned ? half + l * 4 : c + 4;
    const int steps = p.q_steps + p.k_steps + p.v_steps;

    for (int pair = threadIdx.x; pair < half; pair += ROPE_WARPS * 32) units[pair] = turns_per_position(__ldg(p.inv_freq + pair));
    __syncthreads();
    const uint4 none = make_uint4(0, 0, 0, 0);
    auto load_pairs = [&](const __nv_bfloat16* row) {
        if constexpr (HALVES) {
            const uint2 a = *reinterpret_cast<const uint2*>(row + c0), b = *reinterpret_cast<const uint2*>(row + c1);
            return make_uint4(a.x, a.y, b.x, b.y);
        } else {
            return *reinterpret_cast<const uint4*>(row + c);
        }
    };
    auto store_pairs = [&](__nv_bfloat16* row, const uint4& v) {
        if constexpr (HALVES) {
            *reinterpret_cast<uint2*>(row + c0) = make_uint2(v.x, v.y);
            *reinterpret_cast<uint2*>(row + c1) = make_uint2(v.z, v.w);
        } else {
            *reinterpret_cast<uint4*>(row + c) = v;
        }
    };
    const float inv_d = 1.f / float(D);

    // The root mean square's reciprocal; `sum` of a lane's squares.
    auto rstd_of = [&](float sum) {
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        return rsqrtf(fmaf(sum, inv_d, p.eps));
    };

    for (int64_t item = int64_t(blockIdx.x) * ROPE_WARPS + warp; item < p.items; item += int64_t(gridDim.x) * ROPE_WARPS) {
        const int t = p.parts == 1 ? int(item) : int(item / p.parts), part = int(item - int64_t(t) * p.parts);
        const int s0 = int(int64_t(steps) * part / p.parts), s1 = int(int64_t(steps) * (part + 1) / p.parts);

        const int64_t slot = CACHE != MK_CACHE_NONE ? __ldg(p.slots + t) : 0;
        // sines and cosines of the token's pairs
        if (s0 < p.q_steps + p.k_steps && half > 0) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < (PAIRS + 31) / 32; ++i) {
                const int pair = i * 32 + lane;
                if (pair < half) {
                    const int64_t pos = __ldg(p.positions + p.axis[pair] * p.position_stride + t);
                    // the nearest quarter turn and what is left of it, at most an eighth: near a zero
                    // of either function, small angles among them, it keeps 24 bits of its own
                    const uint64_t turn = uint64_t(pos) * units[pair];
                    const uint32_t quarter = uint32_t((turn + (uint64_t(1) << 61)) >> 62);
                    const int64_t left = int64_t(turn - (uint64_t(quarter) << 62));
                    float sine, cosine;
                    sincospif(float(left) * 1.0842021724855044e-19f /* 2^-63 */, &sine, &cosine);
                    if (quarter & 1) {
                        const float c = cosine;
                        cosine = -sine;
                        sine = c;
                    }
                    if (quarter & 2) {
                        cosine = -cosine;
                        sine = -sine;
                    }
                    table[warp][pair] = make_float2(cosine, sine);
                }
            }
            __syncwarp();
        }

        // What the columns of a pair give to the turned pair, weights and angle together:
        // a' = ca (rstd a) + sb (rstd b), b' = cb (rstd b) + sa (rstd a).
        struct Turn {
            float2 ca[2], cb[2], sa[2], sb[2];
        };
        auto turn_of = [&](const __nv_bfloat16* weight) {
            Turn u;
            Pairs f = unpack_pairs<HALVES>(live && weight ? load_pairs(weight) : none);
            float4 e[2];  // cosines and sines of two pairs each
            e[0] = e[1] = make_float4(1.f, 0.f, 1.f, 0.f);
            if (turned) {
                e[0] = *reinterpret_cast<const float4*>(&table[warp][l * 4]);
                e[1] = *reinterpret_cast<const float4*>(&table[warp][l * 4 + 2]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!weight) f.a[i] = f.b[i] = make_float2(1.f, 1.f);
                const float2 cs = make_float2(e[i].x, e[i].z), sn = make_float2(e[i].y, e[i].w);
                u.ca[i] = mul2(f.a[i], cs);
                u.cb[i] = mul2(f.b[i], cs);
                u.sa[i] = mul2(f.a[i], sn);
                u.sb[i] = mul2(f.b[i], make_float2(-sn.x, -sn.y));
            }
            return u;
        };
        auto norm_and_turn = [&](Pairs& y, const void* weight, const Turn& u) {
            float rstd = 1.f;
            if (weight) {
                float2 sum = mul2(y.a[0], y.a[0]);
                sum = fma2(y.a[1], y.a[1], sum);
                sum = fma2(y.b[0], y.b[0], sum);
                sum = fma2(y.b[1], y.b[1], sum);
                rstd = rstd_of(sum.x + sum.y);
            }
            const float2 r = make_float2(rstd, rstd);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 a = mul2(y.a[i], r), b = mul2(y.b[i], r);
                y.a[i] = mul2(a, u.ca[i]);
                y.b[i] = mul2(b, u.cb[i]);
                if (turned) {  // (else an infinite partner would make it NaN)
                    y.a[i] = fma2(b, u.sb[i], y.a[i]);
                    y.b[i] = fma2(a, u.sa[i], y.b[i]);
                }
            }
        };
        // The same of eight neighbouring columns, whose partners another lane holds.
        auto norm_and_turn_in_order = [&](float (&y)[8], const __nv_bfloat16* weight) {
            if (weight) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(y[i], y[i], sum);
                const float rstd = rstd_of(sum);
                float f[8];
                unpack8(live ? __ldg(reinterpret_cast<const uint4*>(weight + c)) : none, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * f[i];
            }
            const int partner = !turned ? lane : c < half ? lane + half / 8 : lane - half / 8;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, y[i], partner);
            if (turned)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 e = table[warp][(c < half ? c : c - half) + i];
                    y[i] = fmaf(o[i], c < half ? -e.y : e.y, y[i] * e.x);
                }
        };
        // Eight neighbouring columns into a 4-bit cache (the lane's place in it); `out`: what
        // it holds of them, or null.
        auto keep = [&](const float (&y)[8], bool on, uint8_t* cache, uint8_t* scales, const float* factor, __nv_bfloat16* out) {
            const float f = factor && on ? __ldg(factor) : 1.f;
            float a = 0.f;
            float2 g[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = make_float2(y[2 * i], y[2 * i + 1]);
                a = max_nan(a, max_nan(fabsf(g[i].x), fabsf(g[i].y)));
            }
            a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
            if (!(a < 3e38f)) {
                // infinite and NaN values: a scale of 448 or NaN, and what is beyond the largest value is that
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    g[i] = make_float2(fminf(fmaxf(g[i].x / f, -1e30f), 1e30f), fminf(fmaxf(g[i].y / f, -1e30f), 1e30f));
                a = fabsf(a / f);
            } else if (factor) {
                const Quotient by(f);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = by.of(g[i]);
                a = fabsf(by.of(a));  // of the largest: the largest
            }
            const uint32_t byte = fp4_scale(a);
            const float scale = float_of_half(halves_of_e4m3x2(byte));
            const Quotient by(scale);
            uint32_t e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = by.of(g[i]);
                e[i] = e2m1x2_of(g[i].x, g[i].y);
            }
            const uint32_t w = __byte_perm(__byte_perm(e[0], e[1], 0x0040), __byte_perm(e[2], e[3], 0x0040), 0x5410);
            if (on && cache) {
                *reinterpret_cast<uint32_t*>(cache) = w;
                if ((l & 1) == 0) *scales = uint8_t(byte);
            }
            if (on && out) {
                const float2 by2 = make_float2(scale, scale), f2 = make_float2(f, f);
                halves_of_e2m1x8(w, e[0], e[1], e[2], e[3]);
                float held[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = mul2(mul2(make_float2(float_of_half(e[i]), float_of_half(e[i] >> 16)), by2), f2);
                    held[2 * i] = v.x;
                    held[2 * i + 1] = v.y;
                }
                *reinterpret_cast<uint4*>(out + c) = pack8(held);
            }
        };

        // The rows of one kind, AHEAD of them on their way at a time; this lane's first one is
        // of head h, `src` its place.
        auto rows = [&](auto ahead, int first, int n, int heads, const __nv_bfloat16* src, int64_t stride, auto&& load, auto&& work) {
            constexpr int AHEAD = decltype(ahead)::value;
            const int a = max(s0 - first, 0), b = min(s1 - first, n);
            int h = a * ROWS + sub;
            src += h * stride;
            for (int s = a; s < b; s += AHEAD) {
                uint4 x[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const bool on = s + i < b && live && h + i * ROWS < heads;
                    x[i] = on ? load(src + i * ROWS * stride) : none;
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (s + i < b) work(h + i * ROWS, live && h + i * ROWS < heads, x[i]);
                h += AHEAD * ROWS;
                src += AHEAD * ROWS * stride;
            }
        };
        using Deep = std::integral_constant<int, ROPE_AHEAD>;
        using Shallow = std::integral_constant<int, CACHE == MK_CACHE_FP4 ? 2 : ROPE_AHEAD>;  // the code of 4 bits is long
        if (s0 < p.q_steps) {
            const Turn u = turn_of(p.q_weight);
            __nv_bfloat16* const out = p.q_out + int64_t(t) * p.Hq * D;
            rows(Deep{}, 0, p.q_steps, p.Hq, p.q + t * p.q_stride, p.q_head, load_pairs, [&](int h, bool on, const uint4& x) {
                Pairs y = unpack_pairs<HALVES>(x);
                norm_and_turn(y, p.q_weight, u);
                if (on) store_pairs(out + h * D, pack_pairs<HALVES>(y));
            });
        }
        if (s1 <= p.q_steps) continue;
        // where the token's keys and values go, or nowhere
        int64_t kept = 0, kept_scales = 0;
        bool stored = false;
        if constexpr (CACHE != MK_CACHE_NONE) {
            stored = slot >= 0 && slot < p.capacity;
            if (slot >= p.capacity && lane == 0) cache_error(p.err, 2u /* fault */, SITE_SLOT_RANGE, uint32_t(t));
            if (stored) {
                const int64_t page = slot < (int64_t(1) << 31) ? int64_t(uint32_t(slot) / uint32_t(p.page_size)) : slot / p.page_size;
                const int64_t token = slot - page * p.page_size;
                kept = page * p.page_stride + token * p.token_stride;
                kept_scales = page * p.scale_page + token * p.scale_token;
            }
        }
        if (s0 < p.q_steps + p.k_steps) {
            __nv_bfloat16* const out = p.k_out ? p.k_out + int64_t(t) * p.Hkv * D : nullptr;
            if constexpr (CACHE == MK_CACHE_FP4) {
                Turn u;
                if constexpr (!KEYS_IN_ORDER) u = turn_of(p.k_weight);
                const auto load = [&](const __nv_bfloat16* row) { return KEYS_IN_ORDER ? *reinterpret_cast<const uint4*>(row + c) : load_pairs(row); };
                rows(Shallow{}, p.q_steps, p.k_steps, p.Hkv, p.k + t * p.k_stride, p.k_head, load, [&](int h, bool on, const uint4& x) {
                    float y[8];
                    if constexpr (KEYS_IN_ORDER) {
                        unpack8(x, y);
                        norm_and_turn_in_order(y, p.k_weight);
                    } else {
                        Pairs z = unpack_pairs<HALVES>(x);
                        norm_and_turn(z, p.k_weight, u);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            y[4 * i] = z.a[i].x;
                            y[4 * i + 1] = z.b[i].x;
                            y[4 * i + 2] = z.a[i].y;
                            y[4 * i + 3] = z.b[i].y;
                        }
                    }
                    keep(y, on, stored ? p.k_cache + kept + h * p.head_stride + c / 2 : nullptr,
                         p.k_scales + kept_scales + h * p.scale_head + c / FP4_GROUP, p.k_factor ? p.k_factor + h : nullptr,
                         out ? out + h * D : nullptr);
                });
            } else {
                const Turn u = turn_of(p.k_weight);
                rows(Deep{}, p.q_steps, p.k_steps, p.Hkv, p.k + t * p.k_stride, p.k_head, load_pairs, [&](int h, bool on, const uint4& x) {
                    Pairs y = unpack_pairs<HALVES>(x);
                    norm_and_turn(y, p.k_weight, u);
                    const uint4 v = pack_pairs<HALVES>(y);
                    if (CACHE == MK_CACHE_BF16 && on && stored)
                        store_pairs(reinterpret_cast<__nv_bfloat16*>(p.k_cache + kept + h * p.head_stride), v);
                    if (on && out) store_pairs(out + h * D, v);
                });
            }
        }
        if constexpr (CACHE != MK_CACHE_NONE) {
            const auto load = [&](const __nv_bfloat16* row) { return *reinterpret_cast<const uint4*>(row + c); };
            __nv_bfloat16* const out = p.v_out ? p.v_out + int64_t(t) * p.Hkv * D : nullptr;
            rows(Shallow{}, p.q_steps + p.k_steps, p.v_steps, p.Hkv, p.v + t * p.v_stride, p.v_head, load, [&](int h, bool on, const uint4& x) {
                if constexpr (CACHE == MK_CACHE_BF16) {  // as they are
                    if (on && stored) *reinterpret_cast<uint4*>(p.v_cache + kept + h * p.head_stride + c * 2) = x;
                } else {
                    float y[8];
                    unpack8(x, y);
                    keep(y, on, stored ? p.v_cache + kept + h * p.head_stride + c / 2 : nullptr,
                         p.v_scales + kept_scales + h * p.scale_head + c / FP4_GROUP, p.v_factor ? p.v_factor + h : nullptr,
                         out ? out + h * D : nullptr);
                }
            });
        }
    }
}

template <int LANES, bool HALVES, int CACHE>
void launch_rope(const RopeParams& p, int grid, cudaStream_t st) {
    if (p.D == LANES * 8 && p.rot == p.D) mk_qk_norm_rope_kernel<LANES, HALVES, CACHE, true><<<grid, ROPE_WARPS * 32, 0, st>>>(p);
    else mk_qk_norm_rope_kernel<LANES, HALVES, CACHE, false><<<grid, ROPE_WARPS * 32, 0, st>>>(p);
}
template <int LANES>
void launch_rope(const RopeParams& p, bool halves, int cache, int grid, cudaStream_t st) {
    if (cache == MK_CACHE_NONE) halves ? launch_rope<LANES, true, MK_CACHE_NONE>(p, grid, st) : launch_rope<LANES, false, MK_CACHE_NONE>(p, grid, st);
    else if (cache == MK_CACHE_BF16) halves ? launch_rope<LANES, true, MK_CACHE_BF16>(p, grid, st) : launch_rope<LANES, false, MK_CACHE_BF16>(p, grid, st);
    else halves ? launch_rope<LANES, true, MK_CACHE_FP4>(p, grid, st) : launch_rope<LANES, false, MK_CACHE_FP4>(p, grid, st);
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
    // A warp per token when there are enough of them; else parts of a token's heads, of
    // four turns or more (each part computes the token's sines), or of one where all of
    // them are at work at once all the same.
    const int64_t warps = int64_t(sms) * ROPE_CTAS * ROPE_WARPS;
    const int64_t most = int64_t(a->T) * steps * 2 <= warps ? steps : (steps + 3) / 4;
    p.parts = int(std::max<int64_t>(1, std::min<int64_t>(most, warps / a->T)));
    p.items = int64_t(a->T) * p.parts;
    const int grid = int(std::min<int64_t>((p.items + ROPE_WARPS - 1) / ROPE_WARPS, int64_t(sms) * ROPE_CTAS));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool halves = a->pairs == MK_PAIR_HALVES;
    if (lanes == 4) launch_rope<4>(p, halves, a->cache, grid, st);
    else if (lanes == 8) launch_rope<8>(p, halves, a->cache, grid, st);
    else if (lanes == 16) launch_rope<16>(p, halves, a->cache, grid, st);
    else launch_rope<32>(p, halves, a->cache, grid, st);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
