// mk_attn4.cu -- mk_paged_attention_fp4: attention of one new token per sequence
// over a paged cache in 4 bits, split over the caches' lengths and joined.
//
//   k = e2m1 * e4m3 scale of its 16 columns * factor of its head, v likewise,
//   s_j = scale * q . k_j,   out = sum_j e^(s_j - m) v_j / l,
//   m = max_j s_j,  l = sum_j e^(s_j - m),  lse = m + log l
//
// A row of 128 columns is 72 bytes, so a key and its value have 6 cycles of an SM
// at the copy rate: the instructions that unpack, scale and multiply 256 values
// bound it as much as the bytes do, and their count decides.
//
// The products have keys (of the scores) or columns (of the output) as their 16
// rows and query heads as their 8 columns, so up to 8 heads waste nothing and 16
// share the unpacked values.  The order of the columns in a score's sum is free:
// a lane takes D/4 neighbouring ones of a key, 16 bytes with 128, and the queries
// are laid out alike.  Of a value it takes D/8 neighbouring columns of four keys;
// pairs of keys are formed while the values have 4 bits.  value * scale has 6
// significant bits and is exact in fp16; the queries keep their 8 there, moved by
// a power of two per head; the weights e^(s - m) are rounded to fp16, 11 bits, an
// eighth of the output's own rounding, and moved by 2^10 so that those above
// 2^-24 of the largest keep all of them (two parts of 11 bits, as exact as fp32,
// cost 16 products and 24 more instructions a tile: 104 us became 117).
//
// Work is cut and joined as in mk_attn_split.cuh.  A tile is KEYS keys of one
// (sequence, group of up to 8, 16 or 24 query heads of one key-value head); each warp
// has a ring of tiles in shared memory, filled by its own asynchronous copies.
//
// Measured on GB300: four sequences of 131071 keys, 8 key-value heads of 128: 104 us,
// 5.8 TB/s (524 instructions a tile of 32 keys, 2.3 a cycle and SM); 64 sequences of 0
// to 16384 keys in pages of 24 (128 MB) 40 us, of which 4 until the first copies and 7
// for the joins; one of 8191 keys 12.0 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mk.h"
#include "mk_attn_split.cuh"
#include "mk_common.h"
#include "mk_fp4.cuh"
#include "mk_host.h"

namespace mk {
namespace {

// What a CTA's ranges have of their first groups, where shared memory has no room
// for it.  Fixed, so the counters never move.
constexpr int ATTN4_HEADS_FLOATS = 34 * 1024;
constexpr size_t ATTN4_HEADS_BYTES = size_t(ATTN_MAX_CTAS) * ATTN4_HEADS_FLOATS * 4;

// D columns a head, groups of NT * 8 query heads.
template <int D, int NT, int UNIT>
struct Geo4 {
    static constexpr int GROUP = NT * 8;
    // Per tile.  (16 sequences of 50000 keys, 12 heads of 64: 130 us with 64, 150 with 32.)
    static constexpr int KEYS = D == 256 ? 16 : D == 64 && NT == 1 && UNIT > 0 ? 64 : 32;
    static constexpr int WARPS = D == 64 ? (NT == 1 ? 16 : NT == 2 ? 12 : 8) : NT == 1 ? 12 : 8;
    static constexpr int STAGES = KEYS == 64 ? 2 : D == 64 ? (NT == 1 ? 4 : 3) : D == 128 ? (NT == 1 ? 2 : 3) : (NT == 1 ? 2 : 4);
    static constexpr int THREADS = WARPS * 32;
    static constexpr int ROW = D / 2;         // bytes of a row's values
    static constexpr int SROW = D / 16;       // bytes of its scales
    static constexpr int VALUES = KEYS * ROW;
    static constexpr int SCALES = KEYS * SROW;
    static constexpr int STAGE = 2 * VALUES + 2 * SCALES;
    static constexpr int RING = STAGES * STAGE;
    static constexpr int PART = GROUP * (D + 8) + 2 * GROUP;  // floats of a range's result: O, m, l
    // The results of ranges' last groups lie where the rings were; those of their first
    // ones beside them, or in the workspace where there is no room.
    // The queries of 16 heads or of 256 columns, laid out for the products, lie in shared
    // memory: in registers they cost spills, which find little L1 beside the rings (13
    // sequences of 47828 keys, 4 heads of 256: 142 us, so 136; 32 of 4096, 8 x 16 heads of
    // 128: 55, so 53).
    static constexpr bool Q_SHARED = NT > 1 || D == 256;
    static constexpr int Q_BYTES = Q_SHARED ? NT * (D / 16) * 2 * 32 * 4 : 0;  // of a warp
    static constexpr bool HEADS_SHARED = WARPS * (RING + PART * 4 + Q_BYTES) <= 215000;
    static constexpr int SM_HEADS = WARPS * RING > WARPS * PART * 4 ? WARPS * RING : WARPS * PART * 4;
    static constexpr int SM_PREFIX = SM_HEADS + (HEADS_SHARED ? WARPS * PART * 4 : 0);
    static constexpr int SM_SMALL = SM_PREFIX + (ATTN_MAX_B + 1) * 4 + 12;
    static constexpr int SM_Q = (SM_SMALL + 128 + 15) / 16 * 16;
    static constexpr int SMEM = SM_Q + WARPS * Q_BYTES;
    static_assert(HEADS_SHARED || WARPS * PART <= ATTN4_HEADS_FLOATS, "the first results fit the workspace");
    static_assert(2 * GROUP + GROUP * D <= ATTN_SLOT_FLOATS, "a partial result fits its slot");
    static_assert(SMEM + 2 * WARPS * 28 + 16 <= 232448, "shared memory of one CTA on sm_103");
};

constexpr float WEIGHT_SHIFT = 10.f;  // weights are 2^10 e^(s - m)
constexpr float OUT = -3e38f;        // a product of a key past the end
constexpr float WEIGHT_MOST = 15.f;   // log2 of the largest: one above starts a new maximum

struct Attn4Params {
    const __nv_bfloat16* q;
    const uint8_t *k, *v, *k_scales, *v_scales;
    const float *k_factor, *v_factor;  // or null
    const int32_t* table;
    const int32_t* lens;
    __nv_bfloat16* out;
    float* lse;                        // or null
    float* slots;
    float* heads;                      // ATTN4_HEADS_FLOATS per CTA
    uint32_t* arrived;
    DevError* err;
    int64_t q_stride;
    int64_t page_stride, token_stride, head_stride;  // bytes
    int64_t scale_page, scale_token, scale_head;     // bytes
    int B, Hq, Hkv, page_size, max_pages, num_pages;
    int per_kv, chunks, groups;
    uint32_t page_units, scale_units;  // strides between pages in 16 bytes (UNIT > 0)
    int page_shift;                    // log2 of page_size, or -1:
    uint32_t page_magic, page_more;    // key / page_size is the high word of key * page_magic, shifted
    float scale2;                      // scale * log2(e)
    uint32_t sixteen, byte;            // 16 and 256

    __device__ float value_factor(int kv) const { return v_factor ? __ldg(v_factor + kv) : 1.f; }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
// One half in both.  LEAN: without an instruction where the multiply can take it so.
template <bool LEAN>
__device__ __forceinline__ uint32_t low_twice(uint32_t h2) {
    if constexpr (!LEAN) return __byte_perm(h2, 0, 0x1010);
    uint32_t r;
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(h2));
    return r;
}
template <bool LEAN>
__device__ __forceinline__ uint32_t high_twice(uint32_t h2) {
    if constexpr (!LEAN) return __byte_perm(h2, 0, 0x3232);
    uint32_t r;
    asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(h2));
    return r;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The first n bytes, then zeros.
__device__ __forceinline__ void copy_part(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, bool ok) {
    if constexpr (BYTES == 16) copy16(dst, src, ok);
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(ok ? BYTES : 0) : "memory");
}
template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (WORDS == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(at);
        w[0] = u.x;
        w[1] = u.y;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(at);
        w[0] = u.x;
        w[1] = u.y;
        w[2] = u.z;
        w[3] = u.w;
    }
}
__device__ __forceinline__ uint32_t load_u16(const uint8_t* at) { return *reinterpret_cast<const uint16_t*>(at); }

// The key of the products' row r, of each 8: an order in which the lanes that read
// shared memory together meet different banks (rows of D/2 bytes lie in order).
template <int D>
__device__ __forceinline__ int key_of(int r) {
    return D == 64 ? int(0x57463120u >> (4 * r) & 7u) : r ^ ((r >> 1) & 1);
}

// UNIT: that many keys of a tile lie in one page, a head's rows one after the other,
// so their copies have one base.  0: every row is looked up by itself.
template <int D, int NT, int UNIT>
__global__ void __launch_bounds__(Geo4<D, NT, UNIT>::THREADS, 1) mk_paged_attention_fp4_kernel(const Attn4Params p) {
    using G = Geo4<D, NT, UNIT>;
    // Shifts and pairs of bytes as multiply-adds, by factors that the compiler does not
    // know: with 8 heads the ALU has most of the work, and the pipe of the multiplies has
    // room (108 us, so 105.7, for 4 x 131071 keys; 150 to 130, so 126, with heads of 64;
    // with 16 heads 155, so 161).
    constexpr bool LEAN = NT == 1;
    const auto shift4 = [&](uint32_t w) { return LEAN ? w * p.sixteen : w << 4; };
    const auto two_bytes = [&](uint32_t lo, uint32_t hi) { return LEAN ? hi * p.byte + lo : __byte_perm(lo, hi, 0x0040); };
    constexpr int KEYS = G::KEYS, GROUP = G::GROUP, MT = KEYS / 16, ROW = G::ROW, SROW = G::SROW;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;  // row and pair of columns of this lane in the products
    uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + G::SM_PREFIX);
    uint32_t* small = reinterpret_cast<uint32_t*>(smem + G::SM_SMALL);
    const uint32_t groups = uint32_t(p.groups);
    count_positions<D, KEYS, G::THREADS>(p, prefix, small);

    const uint32_t total = prefix[p.B] * groups;
    // A position per warp, or two where partial results are large: a shorter range only
    // adds some to join (one sequence of 8191 keys, 8 heads a group: 11.7 us with one, 12.1
    // with two; 16 heads 19.1 and 16.8; 8 of 256 columns 23.2 and 21.1; two of 10000 keys,
    // 24 heads 28.0 and 30.7).
    const uint32_t least = uint32_t(G::WARPS * (NT == 2 || (NT == 1 && D == 256) ? 2 : 1));
    const uint32_t nctas = min(gridDim.x, (total + least - 1) / least);
    if (blockIdx.x >= nctas) return;
    const Cut cut_at(total, nctas);
    const uint32_t start = cut_at.start(blockIdx.x), end = cut_at.start(blockIdx.x + 1);
    const Cut warp_cut(end - start, G::WARPS);
    const uint32_t wstart = start + warp_cut.start(warp), wend = start + warp_cut.start(warp + 1);

    // ---- this warp's ring: loads run STAGES tiles ahead, across groups
    uint8_t* const ring_ptr = smem + warp * G::RING;
    const uint32_t ring = smem_u32(ring_ptr);
    Walk load_walk{wstart, wend, prefix, p.B, groups, false};
    Range lr;
    uint32_t load_tile = 0;
    int load_len = 0;
    bool more = true;
    lr.t1 = 0;
    constexpr int CHUNKS = ROW / 16, PIECES = KEYS * CHUNKS / 32;  // of a row; of a lane
    // The next tile's group and length; false when the range has no more.
    auto next_tile = [&]() -> bool {
        if (!more) return false;
        if (load_tile >= lr.t1) {
            if (!load_walk.next(lr)) return more = false;
            load_len = length_of(p, lr.b);
            load_tile = lr.t0;
            // the group's queries head for L1 while its first tiles do for shared memory
            const int kv = lr.g / p.chunks, head0 = kv * p.per_kv + (lr.g % p.chunks) * GROUP;
            const int heads = min(GROUP, (kv + 1) * p.per_kv - head0);
            const char* q = reinterpret_cast<const char*>(p.q + int64_t(lr.b) * p.q_stride + int64_t(head0) * D);
            for (int i = lane; i < heads * (D / 64); i += 32) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i * 128));
        }
        return true;
    };
    auto slot_of = [&](int key) { return p.page_shift >= 0 ? key >> p.page_shift : int(__umulhi(uint32_t(key), p.page_magic) >> p.page_more); };
    auto good_page = [&](int page) {
        if (page >= 0 && page < p.num_pages) return true;
        attn_error(p.err, SITE_PAGE_RANGE, uint32_t(page));
        return false;
    };
    // UNIT > 0: where the next unit's values and scales are (this lane's first piece of
    // them), the same of the group's page 0, what is left of the page, and the page after
    // it, looked up when it began.  A lane's pieces of a unit's scales: those of its own
    // unit of the tile.
    constexpr int U = UNIT > 0 ? UNIT : KEYS, UNITS = KEYS / U;
    constexpr int UNIT_BYTES = U * ROW, UNIT_PIECES = (UNIT_BYTES + 511) / 512, UNIT_LANES = UNIT_BYTES < 512 ? UNIT_BYTES / 16 : 32;
    constexpr int SCALE_LANES = G::SCALES / 16;  // lanes that copy the keys' scales, and as many the values'
    const int scale_byte = (lane % SCALE_LANES) * 16, scale_unit = lane < 2 * SCALE_LANES ? scale_byte / (U * SROW) : -1;
    const uint8_t* const scales = (lane < SCALE_LANES ? p.k_scales : p.v_scales) + scale_byte % (U * SROW);
    const uint32_t lane_dst = ring + lane * 16;
    const uint8_t *k_at = nullptr, *v_at = nullptr, *s_at = nullptr;
    int64_t head_at = 0, head_scales = 0;
    const int32_t* table = nullptr;
    int page_left = 0, page_next = 0, pages_more = 0;
    bool page_ok = false;
    // Else a lane looks up the row of one key, two tiles before it is copied.
    struct Ahead {
        int page, token, kv;
        bool have, in;
    } ahead[2];
    auto look_up = [&](Ahead& a) {
        a.in = false;
        if (!(a.have = next_tile())) return;
        const int key = int(load_tile) * KEYS + (lane & (KEYS - 1));
        ++load_tile;
        if (key >= load_len) return;
        a.in = true;
        const int slot = slot_of(key);
        a.token = key - slot * p.page_size;
        a.kv = lr.g / p.chunks;
        a.page = __ldg(p.table + int64_t(lr.b) * p.max_pages + slot);
    };
    if constexpr (UNIT == 0) {
        look_up(ahead[0]);
        look_up(ahead[1]);
    }
    uint32_t load_at = 0;  // the stage's place in the ring
    // The next page of the group, from its first key.
    auto enter_page = [&]() {
        page_ok = good_page(page_next);
        const uint32_t page = page_ok ? uint32_t(page_next) : 0u;
        const uint64_t at = uint64_t(page) * p.page_units * 16 + head_at;
        k_at = p.k + at;
        v_at = p.v + at;
        s_at = scales + (uint64_t(page) * p.scale_units * 16 + head_scales);
        page_left = p.page_size;
        if (--pages_more >= 0) page_next = __ldg(++table);
    };
    auto issue = [&]() {
        if constexpr (UNIT > 0) {
            const bool fresh = load_tile >= lr.t1;  // another group
            if (next_tile()) {
                int left = load_len - int(load_tile) * KEYS;  // keys from here to the end
                if (fresh) {
                    const int key = int(load_tile) * KEYS, kv = lr.g / p.chunks, slot = slot_of(key);
                    table = p.table + int64_t(lr.b) * p.max_pages + slot;
                    page_next = __ldg(table);
                    const uint32_t token = uint32_t(key - slot * p.page_size);
                    pages_more = slot_of(load_len - 1) - slot;
                    head_at = kv * p.head_stride + (lane & (UNIT_LANES - 1)) * 16;
                    head_scales = kv * p.scale_head;
                    enter_page();
                    // (of a page of 2^31 - 32 keys: offsets in it pass 32 bits)
                    k_at += uint64_t(token) * ROW;
                    v_at += uint64_t(token) * ROW;
                    s_at += uint64_t(token) * SROW;
                    page_left -= int(token);
                }
#pragma unroll
                for (int u = 0; u < UNITS; ++u) {
                    if (page_left == 0 && left > 0) enter_page();
                    const uint32_t dst = lane_dst + load_at + (UNIT_LANES == 32 ? u * UNIT_BYTES : u / 2 * 512);
                    const bool mine = UNIT_LANES == 32 || lane / UNIT_LANES == u % 2;
                    const uint32_t scale_dst = lane_dst + load_at + 2 * G::VALUES;
                    if (page_ok && left >= U) {
#pragma unroll
                        for (int i = 0; i < UNIT_PIECES; ++i)
                            if (mine) {
                                copy16(dst + i * 512, k_at + i * 512);
                                copy16(dst + G::VALUES + i * 512, v_at + i * 512);
                            }
                        if (scale_unit == u) copy16(scale_dst, s_at);
                    } else {  // zeros past the end, and for a page outside the pool
                        const int rows = page_ok ? left : 0;
#pragma unroll
                        for (int i = 0; i < UNIT_PIECES; ++i)
                            if (mine) {
                                const bool in = (i * 32 + (lane & (UNIT_LANES - 1))) / CHUNKS < rows;
                                copy16(dst + i * 512, in ? k_at + i * 512 : p.k, in);
                                copy16(dst + G::VALUES + i * 512, in ? v_at + i * 512 : p.v, in);
                            }
                        // a piece holds the scales of 16 / SROW keys
                        const int bytes = rows * SROW - scale_byte % (U * SROW);
                        if (scale_unit == u) copy_part(scale_dst, bytes > 0 ? s_at : p.k_scales, max(0, min(16, bytes)));
                    }
                    k_at += UNIT_BYTES;
                    v_at += UNIT_BYTES;
                    s_at += U * SROW;
                    page_left -= U;
                    left -= U;
                }
                ++load_tile;
            }
            copy_commit();
        } else {
            const Ahead a = ahead[0];
            if (a.have) {
                const bool ok = a.in && good_page(a.page);
                const uint32_t ks = ring + load_at, kss = ks + 2 * G::VALUES;
                const int64_t own = ok ? a.page * p.page_stride + a.token * p.token_stride + a.kv * p.head_stride : -1;
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    const int piece = i * 32 + lane, row = piece / CHUNKS, chunk = piece % CHUNKS;
                    const int64_t ro = __shfl_sync(0xffffffffu, own, row);
                    const bool in = ro >= 0;
                    const int64_t at = (in ? ro : 0) + chunk * 16;
                    copy16(ks + piece * 16, p.k + at, in);
                    copy16(ks + G::VALUES + piece * 16, p.v + at, in);
                }
                const int64_t sat = ok ? a.page * p.scale_page + a.token * p.scale_token + a.kv * p.scale_head : 0;
                if (KEYS == 32 || lane < KEYS) {
                    copy_small<SROW>(kss + uint32_t(lane * SROW), p.k_scales + sat, ok);
                    copy_small<SROW>(kss + G::SCALES + uint32_t(lane * SROW), p.v_scales + sat, ok);
                }
            }
            copy_commit();
            ahead[0] = ahead[1];
            look_up(ahead[1]);
        }
        load_at = load_at + G::STAGE == G::RING ? 0u : load_at + G::STAGE;
    };
#pragma unroll
    for (int i = 0; i < G::STAGES; ++i) issue();

    // Where this lane reads: its column's D/8 bytes of key key_of(g), and D/16 bytes of
    // the values of the keys key_of(2c), key_of(2c + 1) and 8 on from these.
    const int kg = key_of<D>(g), va = key_of<D>(2 * c), vb = key_of<D>(2 * c + 1);
    uint32_t at = 0;  // the tile's stage
    Walk walk{wstart, wend, prefix, p.B, groups, false};
    Range r;
    // A group that the range does not hold whole is its first (its result is set aside) or
    // its last (kept in registers until the rings are free).
    __shared__ Range pieces[2 * G::WARPS];
    Range* const mine = pieces + 2 * warp;
    if (lane < 2) mine[lane].tiles = 0;
    __syncwarp();
    bool has_tail = false;
    // Output columns g * D/8 + 2t and + 2t + 1 of heads 8n + 2c and 8n + 2c + 1.
    float o[NT][D / 16][4];
    float m[NT][2], most[NT][2];  // reference of the weights, and what no score may pass
    float2 l[NT], base[NT];       // sums of the weights, and what is added to scores for them

    float* const first_results = G::HEADS_SHARED ? reinterpret_cast<float*>(smem + G::SM_HEADS)
                                                 : p.heads + size_t(blockIdx.x) * ATTN4_HEADS_FLOATS;
    auto put = [&](float* part, int heads) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = n * 8 + 2 * c + i;
                if (g == 0) {
                    part[GROUP * (D + 8) + row] = m[n][i] - WEIGHT_SHIFT;
                    part[GROUP * (D + 8) + GROUP + row] = i ? l[n].y : l[n].x;
                }
                float* to = part + row * (D + 8) + g * (D / 8);
                if (row < heads)
#pragma unroll
                    for (int t = 0; t < D / 16; t += 2)
                        *reinterpret_cast<float4*>(to + 2 * t) =
                            make_float4(o[n][t][i], o[n][t][2 + i], o[n][t + 1][i], o[n][t + 1][2 + i]);
            }
    };

    uint2* const q_shared = reinterpret_cast<uint2*>(smem + G::SM_Q + (G::Q_SHARED ? warp * G::Q_BYTES : 0)) + lane;
    while (walk.next(r)) {
        const int kv = r.g / p.chunks, head0 = kv * p.per_kv + (r.g % p.chunks) * GROUP;
        const int heads = min(GROUP, (kv + 1) * p.per_kv - head0);
        const int len = length_of(p, r.b);
        // Queries as the columns of the products: lane (g, c) holds columns c * D/4 ..
        // of head 8n + g.  A power of two takes a head's largest to 2^14 .. 2^15, and a
        // negative scale's sign goes with it, so that the largest product is the largest
        // score.
        uint32_t qb[G::Q_SHARED ? 1 : NT][D / 16][2];
        float f[NT][2];  // from products to scores in units of log 2; not negative
        const float unit = p.scale2 * (p.k_factor ? __ldg(p.k_factor + kv) : 1.f);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool on = n * 8 + g < heads;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + int64_t(r.b) * p.q_stride + int64_t(head0 + (on ? n * 8 + g : 0)) * D + c * (D / 4));
            uint4 raw[D / 32];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                raw[i] = on ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t u = (&raw[i].x)[j] & 0x7fff7fffu;
                    top = max(top, max(u >> 16, u & 0xffffu));
                }
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the largest's biased exponent; below 2^-112 they move by 2^126, whose inverse is
            // still a normal number (subnormals, from 2^-133 on, to 2^-7 and more); 255: as they are
            const int e = int(top >> 7);
            const int up = e == 255 ? 0 : min(141 - e, 126);
            const float by = copysignf(__uint_as_float(uint32_t(up + 127) << 23), unit);
            const float back = __uint_as_float(uint32_t(127 - up) << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t u = (&raw[i].x)[j];
                    qb[G::Q_SHARED ? 0 : n][2 * i + j / 2][j % 2] = pack_h2(__uint_as_float(u << 16) * by, __uint_as_float(u & 0xffff0000u) * by);
                }
            if constexpr (G::Q_SHARED)
#pragma unroll
                for (int x = 0; x < D / 16; ++x) q_shared[(n * (D / 16) + x) * 32] = make_uint2(qb[0][x][0], qb[0][x][1]);
            f[n][0] = fabsf(unit) * __shfl_sync(0xffffffffu, back, 8 * c);
            f[n][1] = fabsf(unit) * __shfl_sync(0xffffffffu, back, 8 * c + 4);
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][t][i] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n] = base[n] = make_float2(0.f, 0.f);
            most[n][0] = most[n][1] = -INFINITY;
        }

        for (uint32_t t = r.t0; t < r.t1; ++t) {
            const uint8_t *ks = ring_ptr + at, *vs = ks + G::VALUES, *kss = vs + G::VALUES, *vss = kss + G::SCALES;
            const bool cut = len - int(t) * KEYS < KEYS;  // (the tile's end may be 2^31)
            copy_wait<G::STAGES - 1>();
            __syncwarp();

            // ---- scores: 16 keys by 8 heads
            float s[MT][NT][4];
            uint32_t w[MT][2][D / 32], sc[MT][2][D / 64];
            auto load_keys = [&](int mt) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* row = ks + ((mt * 16 + h * 8 + kg) * ROW + c * (D / 8));
                    const uint8_t* srow = kss + ((mt * 16 + h * 8 + kg) * SROW + c * (D / 64));
                    if constexpr (D == 64) {
                        load_words<2>(row, w[mt][h]);
                        sc[mt][h][0] = low_twice<LEAN>(halves_of_e4m3x2(*srow));
                    } else if constexpr (D == 128) {
                        load_words<4>(row, w[mt][h]);
                        const uint32_t two = halves_of_e4m3x2(load_u16(srow));
                        sc[mt][h][0] = low_twice<LEAN>(two);
                        sc[mt][h][1] = high_twice<LEAN>(two);
                    } else {
                        uint32_t a[4], b[4], four[1];
                        load_words<4>(row, a);
                        load_words<4>(row + 16, b);
                        load_words<1>(srow, four);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            w[mt][h][i] = a[i];
                            w[mt][h][4 + i] = b[i];
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t two = halves_of_e4m3x2(four[0] >> (16 * i));
                            sc[mt][h][2 * i] = low_twice<LEAN>(two);
                            sc[mt][h][2 * i + 1] = high_twice<LEAN>(two);
                        }
                    }
                }
            };
            // two products' columns of 16 keys
            auto unpack_keys = [&](int mt, int i, uint32_t (&a)[2][4]) {
                halves_of_e2m1x8(w[mt][0][i], a[0][0], a[0][2], a[1][0], a[1][2]);
                halves_of_e2m1x8(w[mt][1][i], a[0][1], a[0][3], a[1][1], a[1][3]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    a[x][0] = mul_h2(a[x][0], sc[mt][0][i / 2]);
                    a[x][2] = mul_h2(a[x][2], sc[mt][0][i / 2]);
                    a[x][1] = mul_h2(a[x][1], sc[mt][1][i / 2]);
                    a[x][3] = mul_h2(a[x][3], sc[mt][1][i / 2]);
                }
            };
            auto score = [&](int mt, int n, bool first, const uint32_t (&a)[4], uint32_t q0, uint32_t q1) {
                if (first) mma_f16_first(s[mt][n], a, q0, q1);
                else mma_f16(s[mt][n], a, q0, q1);
            };
            if constexpr (G::Q_SHARED) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) load_keys(mt);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t a[MT][2][4];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) unpack_keys(mt, i, a[mt]);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 q = q_shared[(n * (D / 16) + 2 * i + x) * 32];
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) score(mt, n, i == 0 && x == 0, a[mt][x], q.x, q.y);
                        }
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    load_keys(mt);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t a[2][4];
                        unpack_keys(mt, i, a);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int n = 0; n < NT; ++n) score(mt, n, i == 0 && x == 0, a[x], qb[n][2 * i + x][0], qb[n][2 * i + x][1]);
                    }
                }
            }

            // ---- weights
            uint32_t pb[MT][NT][2];
            if (cut) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (int(t) * KEYS + mt * 16 + h * 8 + kg >= len)
#pragma unroll
                            for (int n = 0; n < NT; ++n) s[mt][n][2 * h] = s[mt][n][2 * h + 1] = OUT;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float x0 = s[0][n][0], x1 = s[0][n][1];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    if (mt > 0) {
                        x0 = fmaxf(x0, s[mt][n][0]);
                        x1 = fmaxf(x1, s[mt][n][1]);
                    }
                    x0 = fmaxf(x0, s[mt][n][2]);
                    x1 = fmaxf(x1, s[mt][n][3]);
                }
                x0 *= f[n][0];
                x1 *= f[n][1];
                // The maximum is taken anew only when a weight would pass 2^15 (from nothing: at
                // any score); until then the one before stands for it.
                if (__any_sync(0xffffffffu, x0 > most[n][0] || x1 > most[n][1])) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
                        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
                    }
                    const float n0 = fmaxf(m[n][0], x0), n1 = fmaxf(m[n][1], x1);
                    const float f0 = m[n][0] == -INFINITY ? 0.f : exp2_of(m[n][0] - n0);
                    const float f1 = m[n][1] == -INFINITY ? 0.f : exp2_of(m[n][1] - n1);
                    m[n][0] = n0;
                    m[n][1] = n1;
                    most[n][0] = n0 + (WEIGHT_MOST - WEIGHT_SHIFT);
                    most[n][1] = n1 + (WEIGHT_MOST - WEIGHT_SHIFT);
                    // a head whose scores are all -inf has weights 0, not e^(-inf + inf)
                    base[n] = make_float2(n0 == -INFINITY ? 0.f : WEIGHT_SHIFT - n0, n1 == -INFINITY ? 0.f : WEIGHT_SHIFT - n1);
                    l[n].x *= f0;
                    l[n].y *= f1;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        o[n][j][0] *= f0;
                        o[n][j][1] *= f1;
                        o[n][j][2] *= f0;
                        o[n][j][3] *= f1;
                    }
                }
                float2 w[MT][2];  // of two heads each, by key
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 x = fma2(make_float2(s[mt][n][2 * h], s[mt][n][2 * h + 1]), make_float2(f[n][0], f[n][1]), base[n]);
                        w[mt][h] = make_float2(exp2_of(x.x), exp2_of(x.y));
                    }
                if (cut) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (int(t) * KEYS + mt * 16 + h * 8 + kg >= len) w[mt][h] = make_float2(0.f, 0.f);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        l[n] = add2(l[n], w[mt][h]);
                        pb[mt][n][h] = transpose8(pack_h2(w[mt][h].x, w[mt][h].y));
                    }
            }

            // ---- output: 16 columns by 8 heads, over 16 keys
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                constexpr int WORDS = D / 64;  // of a key's columns here
                uint32_t w[4][WORDS], sb[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = mt * 16 + (j >> 1) * 8 + (j & 1 ? vb : va);
                    load_words<WORDS>(vs + (key * ROW + g * (D / 16)), w[j]);
                    if constexpr (D == 256) sb[j] = load_u16(vss + (key * SROW + 2 * g));
                    else sb[j] = vss[key * SROW + (D == 64 ? g / 2 : g)];
                }
                // scales of the pairs of keys, for the first and the second 16 of the columns
                uint32_t s01[2], s23[2];
                s01[0] = halves_of_e4m3x2(D == 256 ? __byte_perm(sb[0], sb[1], 0x0040) : two_bytes(sb[0], sb[1]));
                s23[0] = halves_of_e4m3x2(D == 256 ? __byte_perm(sb[2], sb[3], 0x0040) : two_bytes(sb[2], sb[3]));
                if constexpr (D == 256) {
                    s01[1] = halves_of_e4m3x2(__byte_perm(sb[0], sb[1], 0x0051));
                    s23[1] = halves_of_e4m3x2(__byte_perm(sb[2], sb[3], 0x0051));
                }
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    constexpr uint32_t LOW = 0x0f0f0f0fu;
                    uint32_t a[4][4];
                    // bytes of one column of two keys
                    halves_of_e2m1x8((w[0][i] & LOW) | (shift4(w[1][i]) & ~LOW), a[0][0], a[1][0], a[2][0], a[3][0]);
                    halves_of_e2m1x8(((w[0][i] >> 4) & LOW) | (w[1][i] & ~LOW), a[0][1], a[1][1], a[2][1], a[3][1]);
                    halves_of_e2m1x8((w[2][i] & LOW) | (shift4(w[3][i]) & ~LOW), a[0][2], a[1][2], a[2][2], a[3][2]);
                    halves_of_e2m1x8(((w[2][i] >> 4) & LOW) | (w[3][i] & ~LOW), a[0][3], a[1][3], a[2][3], a[3][3]);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int half = D == 256 ? i / 2 : 0;
                        a[x][0] = mul_h2(a[x][0], s01[half]);
                        a[x][1] = mul_h2(a[x][1], s01[half]);
                        a[x][2] = mul_h2(a[x][2], s23[half]);
                        a[x][3] = mul_h2(a[x][3], s23[half]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * i + x], a[x], pb[mt][n][0], pb[mt][n][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the tile before it is overwritten
            issue();
            at = at + G::STAGE == G::RING ? 0u : at + G::STAGE;
        }

#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, d);
                l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, d);
            }
        if (r.t1 - r.t0 == r.tiles) {
            // the whole group: straight to the output
            const float factor = p.value_factor(kv);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = n * 8 + 2 * c + i;
                    if (row >= heads) continue;
                    const float sum = i ? l[n].y : l[n].x, inv = sum == 0.f ? 0.f : factor / sum;
                    const int64_t row_at = int64_t(r.b) * p.Hq + head0 + row;
                    uint2* to = reinterpret_cast<uint2*>(p.out + row_at * D + g * (D / 8));
#pragma unroll
                    for (int t = 0; t < D / 16; t += 2)
                        to[t / 2] = make_uint2(pack_bf16(o[n][t][i] * inv, o[n][t][2 + i] * inv),
                                               pack_bf16(o[n][t + 1][i] * inv, o[n][t + 1][2 + i] * inv));
                    if (p.lse && g == 0)
                        p.lse[row_at] = sum == 0.f ? -INFINITY : (m[n][i] - WEIGHT_SHIFT + log2f(sum)) * LN2;
                }
        } else if (walk.pos < walk.end) {
            if (lane == 0) mine[0] = r;
            put(first_results + warp * G::PART, heads);
        } else {
            if (lane == 0) mine[1] = r;
            has_tail = true;
        }
    }
    copy_wait<0>();

    float* tails = reinterpret_cast<float*>(smem);
    __syncthreads();  // the rings are free
    if (has_tail) {
        const int kv = r.g / p.chunks, head0 = kv * p.per_kv + (r.g % p.chunks) * GROUP;
        put(tails + warp * G::PART, min(GROUP, (kv + 1) * p.per_kv - head0));
    }
    join_ranges<D, GROUP, G::WARPS, G::THREADS>(p, pieces, tails, first_results, small, cut_at, start, end);
}

template <int D, int NT, int UNIT>
cudaError_t launch_attn4(Attn4Params& p, int grid, cudaStream_t st) {
    using G = Geo4<D, NT, UNIT>;
    p.chunks = (p.per_kv + G::GROUP - 1) / G::GROUP;
    p.groups = p.chunks * p.Hkv;
    mk_paged_attention_fp4_kernel<D, NT, UNIT><<<grid, G::THREADS, G::SMEM, st>>>(p);
    return cudaGetLastError();
}
template <int D, int NT>
cudaError_t launch_attn4(Attn4Params& p, bool rows, int grid, cudaStream_t st) {
    if (rows && p.page_size % Geo4<D, NT, 16>::KEYS == 0) return launch_attn4<D, NT, Geo4<D, NT, 16>::KEYS>(p, grid, st);
    if (rows && p.page_size % 16 == 0) return launch_attn4<D, NT, 16>(p, grid, st);
    if (rows && p.page_size % 8 == 0) return launch_attn4<D, NT, 8>(p, grid, st);
    return launch_attn4<D, NT, 0>(p, grid, st);
}
// Groups of 8 heads, of 16, or, where that takes fewer passes over the keys and the
// registers are there, of 24 (32 sequences of 4096 keys, 8 key-value heads of 24: 70 us, by
// groups of 16 87; 222 short sequences with one of 24: 21 and 19).
template <int D>
cudaError_t launch_attn4(Attn4Params& p, bool rows, int grid, cudaStream_t st) {
    if (p.per_kv <= 8) return launch_attn4<D, 1>(p, rows, grid, st);
    if constexpr (D < 256)
        if ((p.per_kv + 23) / 24 < (p.per_kv + 15) / 16) return launch_attn4<D, 3>(p, rows, grid, st);
    return launch_attn4<D, 2>(p, rows, grid, st);
}

// Groups of up to 8 query heads per sequence (the smallest), 0 for sizes outside the limits.
int64_t attn4_groups(int B, int Hq, int Hkv) {
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return 0;
    return int64_t(Hkv) * ((Hq / Hkv + 7) / 8);
}

template <int D, int NT, int UNIT>
cudaError_t attn4_smem() {
    return cudaFuncSetAttribute(mk_paged_attention_fp4_kernel<D, NT, UNIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Geo4<D, NT, UNIT>::SMEM);
}
template <int D, int NT>
cudaError_t attn4_smem() {
    for (const cudaError_t e : {attn4_smem<D, NT, Geo4<D, NT, 16>::KEYS>(), attn4_smem<D, NT, 16>(), attn4_smem<D, NT, 8>(), attn4_smem<D, NT, 0>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace

cudaError_t attn4_kernel_attributes() {
    for (const cudaError_t e : {attn4_smem<64, 1>(), attn4_smem<64, 2>(), attn4_smem<64, 3>(), attn4_smem<128, 1>(), attn4_smem<128, 2>(), attn4_smem<128, 3>(),
                                attn4_smem<256, 1>(), attn4_smem<256, 2>()})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_paged_attention_fp4_workspace_size(int B, int Hq, int Hkv) {
    const int64_t g = attn4_groups(B, Hq, Hkv);
    if (g == 0 || B > ATTN_MAX_B) return 0;
    return ATTN_SLOTS_BYTES + ATTN4_HEADS_BYTES + ws_align(size_t(B) * size_t(g) * sizeof(uint32_t));
}

extern "C" mk_status_t mk_paged_attention_fp4(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                              int64_t page_stride, int64_t token_stride, int64_t head_stride,
                                              const void* k_scales, const void* v_scales, int64_t scale_page_stride,
                                              int64_t scale_token_stride, int64_t scale_head_stride, const float* k_factor,
                                              const float* v_factor, const int32_t* block_table, const int32_t* seq_lens,
                                              int B, int Hq, int Hkv, int D, int page_size, int max_pages, int num_pages,
                                              float scale, void* out, float* lse, void* stream, void* workspace,
                                              size_t ws_bytes) {
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || page_size < 1 || max_pages < 0 || num_pages < 0)
        return MK_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return MK_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return MK_ERR_INVALID_ARG;
    const int64_t groups = attn4_groups(B, Hq, Hkv);
    const int64_t cap = int64_t(max_pages) * page_size;
    if (B > ATTN_MAX_B || cap > (int64_t(1) << 31) - 32) return MK_ERR_UNSUPPORTED;
    // positions in the order of tiles are 32-bit
    const int64_t tiles = int64_t(B) * positions_of(int(cap), Geo4<256, 1, 0>::KEYS);
    if (tiles >= int64_t(1) << 31 || tiles * groups >= int64_t(1) << 31) return MK_ERR_UNSUPPORTED;
    if (B > 0) {
        if (!q || !seq_lens || !out) return MK_ERR_INVALID_ARG;
        if (cap > 0 && (!k_cache || !v_cache || !k_scales || !v_scales || !block_table || num_pages < 1)) return MK_ERR_INVALID_ARG;
        const size_t row = size_t(D) / 16;  // scales of a row are copied at once
        if (!host_aligned(q, 16) || !host_aligned(out, 8) || !host_aligned(k_cache, 16) || !host_aligned(v_cache, 16) ||
            !host_aligned(k_scales, row) || !host_aligned(v_scales, row) || !host_aligned(block_table, 4) ||
            !host_aligned(seq_lens, 4) || !host_aligned(lse, 4) || !host_aligned(k_factor, 4) || !host_aligned(v_factor, 4))
            return MK_ERR_INVALID_ARG;
        if (B > 1 && (q_stride < int64_t(Hq) * D || q_stride % 8 != 0)) return MK_ERR_INVALID_ARG;
        // the stride of a dimension of one is never used
        const auto used = [](int n, int64_t s) { return n > 1 ? s : int64_t(0); };
        for (const int64_t v : {used(num_pages, page_stride), used(page_size, token_stride), used(Hkv, head_stride)})
            if (v < 0 || v % 16 != 0) return MK_ERR_INVALID_ARG;
        for (const int64_t v : {used(num_pages, scale_page_stride), used(page_size, scale_token_stride), used(Hkv, scale_head_stride)})
            if (v < 0 || v % int64_t(row) != 0) return MK_ERR_INVALID_ARG;
    }
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    mk_status_t s = host_device(&dev, &sms, &err);
    if (s != MK_OK) return s;
    if (B == 0) return MK_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t need = mk_paged_attention_fp4_workspace_size(B, Hq, Hkv);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Workspace cached;  // held until the launch below
    if (ws) {
        if (ws_bytes < need || !host_aligned(ws, 256)) return MK_ERR_WORKSPACE;
    } else {
        if ((s = cached.get(WS_ATTN4, dev, st, need, need)) != MK_OK) return s;
        ws = cached.data();
    }
    Attn4Params p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const uint8_t*>(k_cache);
    p.v = static_cast<const uint8_t*>(v_cache);
    p.k_scales = static_cast<const uint8_t*>(k_scales);
    p.v_scales = static_cast<const uint8_t*>(v_scales);
    p.k_factor = k_factor;
    p.v_factor = v_factor;
    p.table = block_table;
    p.lens = seq_lens;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.slots = reinterpret_cast<float*>(ws);
    p.heads = reinterpret_cast<float*>(ws + ATTN_SLOTS_BYTES);
    p.arrived = reinterpret_cast<uint32_t*>(ws + ATTN_SLOTS_BYTES + ATTN4_HEADS_BYTES);
    p.err = err;
    p.q_stride = q_stride;
    p.page_stride = page_stride;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.scale_page = scale_page_stride;
    p.scale_token = scale_token_stride;
    p.scale_head = scale_head_stride;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.per_kv = Hq / Hkv;
    p.scale2 = scale * LOG2E;
    p.sixteen = 16;
    p.byte = 256;
    // key / page_size of any key below 2^31 by multiplication (Granlund and Montgomery 1994):
    // with 2^l >= page_size > 2^(l-1), magic = ceil(2^(31+l) / page_size).
    int l = 0;
    while ((int64_t(1) << l) < page_size) ++l;
    p.page_shift = (page_size & (page_size - 1)) == 0 ? l : -1;
    p.page_magic = p.page_shift >= 0 ? 0 : uint32_t(((uint64_t(1) << (31 + l)) + uint32_t(page_size) - 1) / uint32_t(page_size));
    p.page_more = l > 0 ? l - 1 : 0;
    const auto units = [](int n, int64_t s) { return n <= 1 || (s % 16 == 0 && s / 16 <= int64_t(UINT32_MAX)); };
    const bool rows = token_stride == D / 2 && scale_token_stride == D / 16 && host_aligned(k_scales, 16) &&
                      host_aligned(v_scales, 16) && units(num_pages, page_stride) && units(num_pages, scale_page_stride) &&
                      (Hkv <= 1 || scale_head_stride % 16 == 0);
    p.page_units = rows && num_pages > 1 ? uint32_t(page_stride / 16) : 0;
    p.scale_units = rows && num_pages > 1 ? uint32_t(scale_page_stride / 16) : 0;
    const int grid = std::min(sms, ATTN_MAX_CTAS);
    const cudaError_t e = D == 64    ? launch_attn4<64>(p, rows, grid, st)
                          : D == 128 ? launch_attn4<128>(p, rows, grid, st)
                                     : launch_attn4<256>(p, rows, grid, st);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
