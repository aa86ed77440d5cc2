// mk_attn.cu -- mk_paged_attention: attention of one new token per sequence
// over a paged key-value cache, split over the caches' lengths and joined.
//
//   s_j = scale * q . k_j,   out = sum_j e^(s_j - m) v_j / l,
//   m = max_j s_j,  l = sum_j e^(s_j - m),  lse = m + log l
//
// Every key and value is read once for all the query heads that share it, so
// the cache's bytes bound it: 4*D bytes per token and key-value head against
// 4*D operations per query head.
//
// Work.  A tile is 16 keys (32 with 64 columns a head) of one (sequence, group
// of up to 16 or 32 query heads of one key-value head).  The tiles of all of
// them in a row are cut into one equal range per CTA, and that into one per
// warp, whatever the lengths, so every warp streams the same number of bytes
// and waits for no other.  Two warps share a range with 256 columns a head
// (half of the columns each, and they add up their parts of the scores) and in
// groups of 32 heads (16 each, and a ring of tiles).  The caller's lengths stay
// on the device: every CTA builds the table of tiles itself.  A warp writes the
// results of groups that lie whole in its range.  What it has of the others is
// joined in shared memory when the CTA's ranges are done, and what a CTA has of
// groups that it shares with others by the CTA that is done last, in the order
// of the keys.
//
// Each warp has its own ring of tiles in shared memory, filled by its own
// 16-byte asynchronous copies (any page size, any stride, keys past the end
// filled with zeros), which run ahead across the groups of its range.  The
// heads are the rows of m16n8k16 products, so scores and weights stay in
// registers.  tcgen05 wants 64 or 128 rows: keys could be those, not tried; up
// to 16 heads the products take a small part of the time that the bytes do.
//
// Measured on GB300: four sequences of 131071 keys, 8 key-value heads of 128:
// 308 to 317 us, 6.8 to 7.0 TB/s; 13 of 47828 keys, 4 of 256: 360 to 373 us,
// 6.8 to 7.1 TB/s; 64 sequences of 0 to 16384 keys (449 MB) 80 us, of which 67
// until the last keys are in; one of 8191 keys 13.9 us (latency).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mk.h"
#include "mk_common.h"
#include "mk_host.h"
#include "mk_ptx.cuh"

namespace mk {
namespace {

constexpr int ROWS = 16;          // query heads per warp (rows of the product)
// A group counts as this many tiles more than it has: its queries, its first
// tile's latency and its result cost about that, and short groups would
// otherwise gather in a few warps.
constexpr uint32_t EXTRA = 3;
constexpr int ATTN_MAX_B = 4096;  // sequences (their tile counts sit in shared memory)
constexpr int ATTN_MAX_CTAS = 160;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// D columns a head, groups of R * 16 query heads.
template <int D, int R>
struct Geo {
    static constexpr int WARPS = 8;
    static constexpr int GROUP = R * ROWS;
    // Warps that share a range, each with an equal part of the columns: one warp with
    // all 256 leaves room for four rings, a warp per scheduler, and its own latencies
    // bound it (13 sequences of 47828 keys, 4 heads of 256: 547 us, with two 360 to
    // 373).  With 128 columns two warps gain nothing on long sequences (90 us either
    // way) and lose on many short ones (222 of 0 to 1518 keys, 24 heads each: 76, 93).
    static constexpr int SPLIT = D == 256 ? 2 : 1;
    // Warps that share a range: with R = 2 a ring of tiles too, with 16 heads each.
    static constexpr int MATES = SPLIT * R;
    static_assert(MATES <= 2, "they meet in pairs");
    static constexpr int RANGES = WARPS / MATES;
    static constexpr int COLS = D / SPLIT;            // columns of a warp
    static constexpr int STAGES = 2 * R;
    static constexpr int KEYS = D == 64 ? 32 : 16;    // keys per tile
    static constexpr int THREADS = WARPS * 32;
    static constexpr int CHUNKS = COLS / 8;           // 16-byte pieces of a row's part
    static constexpr int HALF = KEYS * COLS * 2;      // a warp's part of one tile's keys (or values)
    static constexpr int RING = STAGES * 2 * HALF;    // of R warps
    static constexpr int OSTRIDE = D + 8;             // floats between rows of the join buffer: no bank conflicts
    // The result of a range's first group and of its last: O, m, l.  The last ones
    // lie where the rings were.
    static constexpr int PART = GROUP * OSTRIDE + 2 * GROUP;
    static constexpr int SM_HEADS = WARPS / R * RING;
    static constexpr int SM_PREFIX = SM_HEADS + RANGES * PART * 4;
    static constexpr int SM_SMALL = SM_PREFIX + (ATTN_MAX_B + 1) * 4 + 12;
    static constexpr int SM_SCORES = SM_SMALL + 128;  // partial scores of warps that share a range, twice
    static constexpr int SMEM = SM_SCORES + (SPLIT > 1 ? 2 * WARPS * (KEYS / 8) * 512 : 0);
    static_assert(RANGES * PART * 4 <= SM_HEADS, "the last results lie where the rings were");
    static constexpr int SLOT = 2 * GROUP + GROUP * D;  // floats of a partial result: m, l, O
    static_assert(SMEM + 2 * RANGES * 24 <= 232448, "shared memory of one CTA on sm_103");
};

constexpr size_t ATTN_SLOT_BYTES = size_t(std::max(Geo<256, 1>::SLOT, Geo<128, 2>::SLOT)) * 4;
constexpr size_t ATTN_SLOTS_BYTES = 2 * ATTN_MAX_CTAS * ATTN_SLOT_BYTES;  // fixed, so the counters never move

struct AttnParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const int32_t* table;
    const int32_t* lens;
    __nv_bfloat16* out;
    float* lse;                                   // or null
    float* slots;                                 // two partial results per CTA
    uint32_t* arrived;                            // per (sequence, group); zero between calls
    DevError* err;
    int64_t q_stride, page_stride, token_stride, head_stride;
    int B, Hq, Hkv, page_size, max_pages, num_pages;
    int per_kv;                                   // query heads per key-value head
    int chunks;                                   // groups per key-value head
    int groups;                                   // groups per sequence
    float scale2;                                 // scale * log2(e)
};

__device__ __forceinline__ void attn_error(DevError* e, uint32_t site, uint32_t info) {
    if (atomicCAS(&e->code, 0u, uint32_t(ERR_FAULT)) == 0u) {
        e->site = site;
        e->cta = blockIdx.x;
        e->info = info;
    }
}

// The two warps of a range meet, and see what each has written and copied.
__device__ __forceinline__ void pair_sync(int range) { asm volatile("bar.sync %0, 64;" ::"r"(1 + range) : "memory"); }

// 16 bytes global -> shared; zeros when !ok (the source is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
// The hardware's exponential, off by 2^-22 of its value at most: a sixty-fourth of
// what the weights lose in the products below.
__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two weights as the sum of two bf16 values each: 16 significant bits reach the
// products (the sum of the weights is of all 24), a 256th of the output's own
// rounding, where one bf16 value would be as coarse as that.  The first is the
// weight cut off; the second, what remains and 2^-23 of the weight, is above 0
// for every weight above 2^-110, so both products with an infinite value are
// infinite, of its sign (rounded to nearest, the remainder may be 0 or negative,
// and the sum of the products NaN).
__device__ __forceinline__ void split_weights(float p0, float p1, uint32_t& hi, uint32_t& lo) {
    const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
    constexpr float ABOVE = 1.f + 1.1920928955078125e-7f;
    hi = __byte_perm(u0, u1, 0x7632);
    lo = pack_bf16(fmaf(p0, ABOVE, -__uint_as_float(u0 & 0xffff0000u)), fmaf(p1, ABOVE, -__uint_as_float(u1 & 0xffff0000u)));
}

// Tiles [t0, t1) of group g of sequence b.  In the order of positions that is
// cut into ranges, EXTRA positions stand before a group's first tile.
struct Range {
    int b, g;
    uint32_t t0, t1;
    uint32_t begin;  // position of the group's first tile
    uint32_t tiles;  // tiles of the group
};
__host__ __device__ inline uint32_t positions_of(int len, int keys) {
    return len > 0 ? uint32_t(len + keys - 1) / uint32_t(keys) + EXTRA : 0u;
}

// The groups of the positions [pos, end) one after the other.
struct Walk {
    uint32_t pos, end;
    const uint32_t* prefix;
    int B;
    uint32_t groups;
    bool started;
    // The next group that has tiles there.
    __device__ bool next(Range& r) {
        do {
            if (pos >= end) return false;
            uint32_t in = 0;  // position inside the group
            if (!started) {
                started = true;
                const uint32_t want = pos / groups;  // positions of one group before it
                int lo = 0, hi = B;                  // the last b with prefix[b] <= want that has keys
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (prefix[mid] <= want) lo = mid;
                    else hi = mid;
                }
                const uint32_t n = prefix[lo + 1] - prefix[lo];
                in = pos - prefix[lo] * groups;
                r.b = lo;
                r.g = int(in / n);
                in -= uint32_t(r.g) * n;
                r.tiles = n - EXTRA;
            } else if (uint32_t(++r.g) == groups) {
                // the next sequence that has keys
                r.g = 0;
                do ++r.b;
                while (prefix[r.b + 1] == prefix[r.b]);
                r.tiles = prefix[r.b + 1] - prefix[r.b] - EXTRA;
            }
            const uint32_t to = min(r.tiles + EXTRA, in + (end - pos));
            r.begin = pos - in + EXTRA;
            r.t0 = in > EXTRA ? in - EXTRA : 0u;
            r.t1 = to > EXTRA ? to - EXTRA : 0u;
            pos += to - in;
        } while (r.t1 <= r.t0);
        return true;
    }
};

// `total` positions cut into n ranges that differ by one position at most:
// the first `more` of them hold `each` + 1.
struct Cut {
    uint32_t each, more;
    __device__ Cut(uint32_t total, uint32_t n) : each(total / n), more(total - (total / n) * n) {}
    __device__ uint32_t start(uint32_t c) const { return c * each + min(c, more); }
    __device__ uint32_t owner(uint32_t p) const {
        const uint32_t in_more = more * (each + 1);
        return p < in_more ? p / (each + 1) : more + (p - in_more) / each;
    }
};

// Element offset of one key's row of a tile (row = lane, modulo the tile's
// keys), or -1 when the key lies past the sequence.
template <int KEYS>
__device__ __forceinline__ int64_t key_offset(const AttnParams& p, int b, int kv, uint32_t tile, int lane, int len) {
    const int key = int(tile) * KEYS + (lane & (KEYS - 1));
    if (key >= len) return -1;
    const int slot = key / p.page_size;
    const int page = __ldg(p.table + int64_t(b) * p.max_pages + slot);
    if (page < 0 || page >= p.num_pages) {
        attn_error(p.err, SITE_PAGE_RANGE, uint32_t(page));
        return -1;
    }
    return page * p.page_stride + (key - slot * p.page_size) * p.token_stride + kv * p.head_stride;
}

// A warp's result of a group: its columns of O, m, l.
template <typename G>
__device__ __forceinline__ void put_partial(float* part, int heads, int row0, int side, const float (&o)[G::COLS / 8][4],
                                            float m0, float m1, float l0, float l1) {
    constexpr int stride = G::OSTRIDE;
    const int lane = threadIdx.x & 31, r0 = lane >> 2, r1 = r0 + 8;
    float* sm = part + G::GROUP * stride + row0;
    if (side == 0 && (lane & 3) == 0) {
        sm[r0] = m0;
        sm[r1] = m1;
        sm[G::GROUP + r0] = l0;
        sm[G::GROUP + r1] = l1;
    }
    float* ow = part + row0 * stride + side * G::COLS + (lane & 3) * 2;
#pragma unroll
    for (int n = 0; n < G::COLS / 8; ++n) {
        if (r0 < heads) *reinterpret_cast<float2*>(ow + r0 * stride + n * 8) = make_float2(o[n][0], o[n][1]);
        if (r1 < heads) *reinterpret_cast<float2*>(ow + r1 * stride + n * 8) = make_float2(o[n][2], o[n][3]);
    }
}

// Four columns of a head's partial result: maximum (in units of log 2), sum of
// weights, weighted sum of values.
struct Part {
    float m = -INFINITY, l = 0.f;
    float4 o = {0.f, 0.f, 0.f, 0.f};

    __device__ void load(const float* slot, int group, int row, int c, int D) {
        m = __ldcg(slot + row);
        l = __ldcg(slot + group + row);
        o = __ldcg(reinterpret_cast<const float4*>(slot + 2 * group + row * D + c));
    }
    template <int N>
    __device__ void add(const Part (&u)[N]) {
        float top = m;
#pragma unroll
        for (int x = 0; x < N; ++x) top = fmaxf(top, u[x].m);
        const float base = top == -INFINITY ? 0.f : top;
        const float f = exp2_of(m - base);
        m = top;
        l *= f;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const float g = exp2_of(u[x].m - base);
            l = fmaf(g, u[x].l, l);
            o.x = fmaf(g, u[x].o.x, o.x);
            o.y = fmaf(g, u[x].o.y, o.y);
            o.z = fmaf(g, u[x].o.z, o.z);
            o.w = fmaf(g, u[x].o.w, o.w);
        }
    }
    __device__ void finish(const AttnParams& p, int b, int head, int c, int D) const {
        const int64_t at = int64_t(b) * p.Hq + head;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<uint2*>(p.out + at * D + c) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (p.lse && c == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
};

// The result of a group from the partial results of CTAs [c0, c0 + n), by a
// whole CTA.  A thread takes four columns of one head and, where there are more threads than
// that, every parts-th piece; the parts are joined in shared memory.
template <int D, int R>
__device__ void join_group(const AttnParams& p, const Range& r, uint32_t c0, int n, uint32_t which0, float* smem_f) {
    using G = Geo<D, R>;
    const int tid = threadIdx.x;
    const int kv = r.g / p.chunks, head0 = kv * p.per_kv + (r.g % p.chunks) * G::GROUP;
    const int heads = min(G::GROUP, (kv + 1) * p.per_kv - head0);
    const int items = heads * (D / 4), parts = min(n, max(1, G::THREADS / items));
    Part* red = reinterpret_cast<Part*>(smem_f);
    // the first CTA's piece may lie in its second slot; the others' ranges start in the group
    const float* first = p.slots + size_t(2 * c0 + which0) * (ATTN_SLOT_BYTES / 4);
    const float* other = p.slots + size_t(2 * c0) * (ATTN_SLOT_BYTES / 4);
    for (int i0 = 0; i0 < items; i0 += G::THREADS) {
        const int item = parts > 1 ? tid % items : i0 + tid, part = parts > 1 ? tid / items : 0;
        const bool on = item < items && part < parts;
        const int row = item / (D / 4), c = (item % (D / 4)) * 4;
        Part acc;
        if (on) {
            constexpr int BATCH = 4;
            for (int i = part; i < n; i += BATCH * parts) {
                Part u[BATCH];
#pragma unroll
                for (int x = 0; x < BATCH; ++x) {
                    const int at = i + x * parts;
                    if (at < n) u[x].load(at == 0 ? first : other + size_t(2 * at) * (ATTN_SLOT_BYTES / 4), G::GROUP, row, c, D);
                }
                acc.add(u);
            }
        }
        if (parts > 1) {
            if (on) red[part * items + item] = acc;
            __syncthreads();
            if (on && part == 0)
                for (int q = 1; q < parts; ++q) {
                    const Part u[1] = {red[q * items + item]};
                    acc.add(u);
                }
        }
        if (on && part == 0) acc.finish(p, r.b, head0 + row, c, D);
    }
    __syncthreads();  // the buffer is free for another group
}

template <int D, int R>
__global__ void __launch_bounds__(Geo<D, R>::THREADS, 1) mk_paged_attention_kernel(const AttnParams p) {
    using G = Geo<D, R>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + G::SM_PREFIX);
    uint32_t* small = reinterpret_cast<uint32_t*>(smem + G::SM_SMALL);
    const uint32_t groups = uint32_t(p.groups);
    const int64_t cap = int64_t(p.max_pages) * p.page_size;

    // ---- positions of one group of each sequence, summed over the sequences before it
    auto length = [&](int b) -> int {
        const int n = __ldg(p.lens + b);
        return n < 0 ? 0 : n > cap ? int(cap) : n;
    };
    {
        const int per = (p.B + G::THREADS - 1) / G::THREADS;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        uint32_t mine = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = __ldg(p.lens + b);
            if ((n < 0 || n > cap) && blockIdx.x == 0) attn_error(p.err, SITE_SEQ_LEN, uint32_t(n));
            mine += positions_of(length(b), G::KEYS);
        }
        uint32_t run = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d) run += o;
        }
        if (lane == 31) small[warp] = run;
        __syncthreads();
        uint32_t base = run - mine;
        for (int w = 0; w < warp; ++w) base += small[w];
        for (int b = b0; b < b1; ++b) {
            prefix[b] = base;
            base += positions_of(length(b), G::KEYS);
        }
        if (b1 == p.B && b0 < b1) prefix[p.B] = base;
        __syncthreads();
    }

    // sequences without keys: zeros and -inf
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (prefix[b + 1] != prefix[b]) continue;
        uint2* o = reinterpret_cast<uint2*>(p.out + int64_t(b) * p.Hq * D);
        for (int i = tid; i < p.Hq * D / 4; i += G::THREADS) o[i] = make_uint2(0u, 0u);
        if (p.lse)
            for (int i = tid; i < p.Hq; i += G::THREADS) p.lse[int64_t(b) * p.Hq + i] = -INFINITY;
    }

    const uint32_t total = prefix[p.B] * groups;
    // At least a position per range, and one more for every four heads of a warp
    // beyond the first four: a shorter range only adds partial results to join
    // (10 sequences, 16 heads, up to 12043 keys: 34 us with one position, 21 with
    // four; 16 sequences of one head a group: 12 us with one, 16 with four).
    const uint32_t least = uint32_t(G::RANGES * max(1, min(ROWS, p.per_kv) / 4));
    const uint32_t nctas = min(gridDim.x, (total + least - 1) / least);
    if (blockIdx.x >= nctas) return;
    const Cut cut_at(total, nctas);
    const uint32_t start = cut_at.start(blockIdx.x), end = cut_at.start(blockIdx.x + 1);
    // this warp's range, its place there, its part of the columns and its first head of a group
    const int range = warp / G::MATES, mate = warp % G::MATES;
    const int side = G::SPLIT > 1 ? mate : 0, row0 = R > 1 ? mate * ROWS : 0;
    const Cut warp_cut(end - start, G::RANGES);
    const uint32_t wstart = start + warp_cut.start(range), wend = start + warp_cut.start(range + 1);
    const __nv_bfloat16 *my_q = p.q + side * G::COLS, *my_k = p.k + side * G::COLS, *my_v = p.v + side * G::COLS;

    // ---- this warp's ring: loads run STAGES tiles ahead, across groups
    const uint32_t ring = smem_u32(smem) + uint32_t(warp / R) * G::RING;
    Walk load_walk{wstart, wend, prefix, p.B, groups, false};
    uint32_t load_tile = 0;
    Range lr;
    int load_len = 0;
    bool more = true;
    lr.t1 = 0;
    // The pages of the next two tiles are looked up before their rows are copied.
    int64_t off[2];   // this lane's row offsets
    bool have[2];
    auto look_up = [&](int64_t& o, bool& h) {
        h = false;
        if (!more) return;
        if (load_tile >= lr.t1) {
            if (!load_walk.next(lr)) {
                more = false;
                return;
            }
            load_len = length(lr.b);
            load_tile = lr.t0;
            // the group's queries head for L1 while its first tiles do for shared memory
            const int head = lr.g / p.chunks * p.per_kv + lr.g % p.chunks * G::GROUP + row0 + (lane & (ROWS - 1));
            if (lane < ROWS && head < (lr.g / p.chunks + 1) * p.per_kv) {
                const char* q = reinterpret_cast<const char*>(my_q + int64_t(lr.b) * p.q_stride + int64_t(head) * D);
#pragma unroll
                for (int i = 0; i < G::COLS * 2; i += 128) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + i));
            }
        }
        o = key_offset<G::KEYS>(p, lr.b, lr.g / p.chunks, load_tile, lane, load_len);
        h = true;
        ++load_tile;
    };
    look_up(off[0], have[0]);
    look_up(off[1], have[1]);
    uint32_t load_slot = 0;
    auto issue = [&]() {
        if (have[0]) {
            const uint32_t dst = ring + load_slot * (2 * G::HALF);
#pragma unroll
            for (int i = 0; i < G::KEYS * G::CHUNKS / (32 * R); ++i) {
                const int piece = (i * R + (R > 1 ? mate : 0)) * 32 + lane, row = piece / G::CHUNKS, c = piece % G::CHUNKS;
                const int64_t ro = __shfl_sync(0xffffffffu, off[0], row);
                const bool ok = ro >= 0;
                const int64_t at = (ok ? ro : 0) + c * 8;
                const uint32_t d = dst + uint32_t(row * G::COLS * 2 + ((c ^ (row & 7)) << 4));
                copy16(d, my_k + at, ok);
                copy16(d + G::HALF, my_v + at, ok);
            }
        }
        copy_commit();
        off[0] = off[1];
        have[0] = have[1];
        look_up(off[1], have[1]);
        if (++load_slot == G::STAGES) load_slot = 0;
    };
    // With a ring of its own a warp refills a stage when it has used it; two warps
    // meet before each tile, so the stage before is free then.
#pragma unroll
    for (int i = 0; i < G::STAGES - (R > 1); ++i) issue();

    const int r0 = lane >> 2, r1 = r0 + 8;  // this lane's rows (heads) of the products
    uint32_t slot = 0, turn = 0;
    Walk walk{wstart, wend, prefix, p.B, groups, false};
    Range r;
    // A group that the range does not hold whole is its first (set aside in shared
    // memory) or its last (kept in registers until the rings are free).
    Range head, tail;
    bool has_head = false, has_tail = false;
    float o[G::COLS / 8][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    while (walk.next(r)) {
        const int kv = r.g / p.chunks, head0 = kv * p.per_kv + (r.g % p.chunks) * G::GROUP + row0;
        const int heads = min(ROWS, (kv + 1) * p.per_kv - head0);  // none or fewer for a second warp
        const int len = length(r.b);
        // query rows as A fragments
        uint32_t qa[G::COLS / 16][4];
        {
            const __nv_bfloat16* qb = my_q + int64_t(r.b) * p.q_stride + int64_t(head0) * D + (lane & 3) * 2;
            const uint32_t* q0 = reinterpret_cast<const uint32_t*>(qb + int64_t(r0 < heads ? r0 : 0) * D);
            const uint32_t* q1 = reinterpret_cast<const uint32_t*>(qb + int64_t(r1 < heads ? r1 : 0) * D);
#pragma unroll
            for (int kk = 0; kk < G::COLS / 16; ++kk) {
                qa[kk][0] = r0 < heads ? q0[kk * 8] : 0u;
                qa[kk][1] = r1 < heads ? q1[kk * 8] : 0u;
                qa[kk][2] = r0 < heads ? q0[kk * 8 + 4] : 0u;
                qa[kk][3] = r1 < heads ? q1[kk * 8 + 4] : 0u;
            }
        }
#pragma unroll
        for (int n = 0; n < G::COLS / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;

        for (uint32_t t = r.t0; t < r.t1; ++t) {
            if constexpr (R > 1) {
                // both warps' copies of the tile are in, and both have used the one before
                copy_wait<G::STAGES - 2>();
                pair_sync(range);
                issue();
            } else {
                copy_wait<G::STAGES - 1>();
                __syncwarp();
            }
            const uint32_t ks = ring + slot * (2 * G::HALF), vs = ks + G::HALF;
            // scores: keys in tiles of 8
            constexpr int NT = G::KEYS / 8;
            float s[NT][4] = {};
            {
                const int row = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
                const uint32_t rb = ks + uint32_t(row * G::COLS * 2);
#pragma unroll
                for (int kk = 0; kk < G::COLS / 16; ++kk) {
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t kb[4];
                        ldsm4(rb + n * 8 * G::COLS * 2 + (uint32_t((kk * 2 + half) ^ (row & 7)) << 4), kb);
                        mma16816(s[n], qa[kk], kb[0], kb[1]);
                        mma16816(s[n + 1], qa[kk], kb[2], kb[3]);
                    }
                }
            }
            if constexpr (G::SPLIT == 2) {
                // the other warp's columns: both add the same two sums, and have all else alike
                float4* at = reinterpret_cast<float4*>(smem + G::SM_SCORES) + turn * (G::WARPS * NT * 32) + lane;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    at[(warp * NT + n) * 32] = make_float4(s[n][0], s[n][1], s[n][2], s[n][3]);
                pair_sync(range);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 u = at[((warp ^ 1) * NT + n) * 32];
                    s[n][0] += u.x;
                    s[n][1] += u.y;
                    s[n][2] += u.z;
                    s[n][3] += u.w;
                }
                turn ^= 1u;  // the next tile's go beside these: one barrier a tile
            }
            const int key = int(t) * G::KEYS + (lane & 3) * 2;
            const bool cut = int(t + 1) * G::KEYS > len;
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][i] *= p.scale2;
                    if (cut && key + n * 8 + (i & 1) >= len) s[n][i] = -INFINITY;
                }
                x0 = fmaxf(x0, fmaxf(s[n][0], s[n][1]));
                x1 = fmaxf(x1, fmaxf(s[n][2], s[n][3]));
            }
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
            if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
                // a new maximum: what was summed so far shrinks (from nothing: stays 0)
                const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                const float f0 = m0 == -INFINITY ? 0.f : exp2_of(m0 - n0);
                const float f1 = m1 == -INFINITY ? 0.f : exp2_of(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int n = 0; n < G::COLS / 8; ++n) {
                    o[n][0] *= f0;
                    o[n][1] *= f0;
                    o[n][2] *= f1;
                    o[n][3] *= f1;
                }
            }
            // a row whose scores are all -inf has weights 0, not e^(-inf + inf)
            const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
            for (int kk = 0; kk < NT / 2; ++kk) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float(&sn)[4] = s[2 * kk + n];
                    const float p0 = exp2_of(sn[0] - b0), p1 = exp2_of(sn[1] - b0);
                    const float p2 = exp2_of(sn[2] - b1), p3 = exp2_of(sn[3] - b1);
                    l0 += p0 + p1;
                    l1 += p2 + p3;
                    split_weights(p0, p1, hi[2 * n], lo[2 * n]);
                    split_weights(p2, p3, hi[2 * n + 1], lo[2 * n + 1]);
                }
                const int row = kk * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
                const uint32_t rb = vs + uint32_t(row * G::COLS * 2);
#pragma unroll
                for (int n = 0; n < G::COLS / 16; ++n) {
                    uint32_t vb[4];
                    ldsm4_t(rb + (uint32_t((n * 2 + half) ^ (row & 7)) << 4), vb);
                    mma16816(o[2 * n], hi, vb[0], vb[1]);
                    mma16816(o[2 * n + 1], hi, vb[2], vb[3]);
                    mma16816(o[2 * n], lo, vb[0], vb[1]);
                    mma16816(o[2 * n + 1], lo, vb[2], vb[3]);
                }
            }
            if constexpr (R == 1) {
                __syncwarp();  // every lane has read the tile before it is overwritten
                issue();
            }
            if (++slot == G::STAGES) slot = 0;
        }

        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (r.t1 - r.t0 == r.tiles) {
            // the whole group: straight to the output
            const float i0 = l0 == 0.f ? 0.f : 1.f / l0, i1 = l1 == 0.f ? 0.f : 1.f / l1;
            const int64_t at = int64_t(r.b) * p.Hq + head0;
            uint32_t* w0 = reinterpret_cast<uint32_t*>(p.out + (at + r0) * D + side * G::COLS) + (lane & 3);
            uint32_t* w1 = reinterpret_cast<uint32_t*>(p.out + (at + r1) * D + side * G::COLS) + (lane & 3);
#pragma unroll
            for (int n = 0; n < G::COLS / 8; ++n) {
                if (r0 < heads) w0[n * 4] = pack_bf16(o[n][0] * i0, o[n][1] * i0);
                if (r1 < heads) w1[n * 4] = pack_bf16(o[n][2] * i1, o[n][3] * i1);
            }
            if (p.lse && side == 0 && (lane & 3) == 0) {
                if (r0 < heads) p.lse[at + r0] = l0 == 0.f ? -INFINITY : (m0 + log2f(l0)) * LN2;
                if (r1 < heads) p.lse[at + r1] = l1 == 0.f ? -INFINITY : (m1 + log2f(l1)) * LN2;
            }
        } else if (walk.pos < walk.end) {
            head = r;
            has_head = true;
            put_partial<G>(reinterpret_cast<float*>(smem + G::SM_HEADS) + range * G::PART, heads, row0, side, o, m0, m1, l0,
                           l1);
        } else {
            tail = r;
            has_tail = true;
        }
    }
    copy_wait<0>();

    // ---- join what the CTA's ranges have of the same groups
    __shared__ Range pieces[2 * G::RANGES];  // in the order of positions; tiles 0: none
    __syncthreads();  // the rings are free
    if (mate == 0 && lane == 0) {
        head.tiles = has_head ? head.tiles : 0u;
        tail.tiles = has_tail ? tail.tiles : 0u;
        pieces[2 * range] = head;
        pieces[2 * range + 1] = tail;
    }
    float* tails = reinterpret_cast<float*>(smem);
    const float* firsts = reinterpret_cast<const float*>(smem + G::SM_HEADS);
    if (has_tail) {
        const int kv = tail.g / p.chunks, head0 = kv * p.per_kv + (tail.g % p.chunks) * G::GROUP + row0;
        put_partial<G>(tails + range * G::PART, min(ROWS, (kv + 1) * p.per_kv - head0), row0, side, o, m0, m1, l0, l1);
    }
    __syncthreads();
    Range open[2];  // groups shared with other CTAs: the first and the last one's
    int nopen = 0;
    uint32_t left = 0;  // pieces not joined yet, a bit each
#pragma unroll
    for (int i = 0; i < 2 * G::RANGES; ++i) left |= pieces[i].tiles != 0 ? 1u << i : 0u;
    while (left) {
        const Range q = pieces[__ffs(int(left)) - 1];
        uint32_t same = 0;  // those of the first one's group
#pragma unroll
        for (int i = 0; i < 2 * G::RANGES; ++i)
            if ((left >> i & 1u) && pieces[i].begin == q.begin) same |= 1u << i;
        left &= ~same;
        const int kv = q.g / p.chunks, head0 = kv * p.per_kv + (q.g % p.chunks) * G::GROUP;
        const int heads = min(G::GROUP, (kv + 1) * p.per_kv - head0);
        const bool whole = q.begin >= start && q.begin + q.tiles <= end;
        // a CTA's first shared group takes its first slot, its last one the second
        float* mine = p.slots + size_t(2 * blockIdx.x + (start >= q.begin ? 0 : 1)) * (ATTN_SLOT_BYTES / 4);
        for (int item = tid; item < heads * (D / 4); item += G::THREADS) {
            const int row = item / (D / 4), c = (item % (D / 4)) * 4;
            Part acc;
            for (uint32_t rest = same; rest;) {
                constexpr int BATCH = 4;
                Part u[BATCH];
#pragma unroll
                for (int x = 0; x < BATCH; ++x) {
                    if (rest == 0) continue;
                    const int i = __ffs(int(rest)) - 1, w = i >> 1;
                    rest &= rest - 1;
                    const float* s = (i & 1 ? tails : firsts) + w * G::PART;
                    u[x].m = s[G::GROUP * G::OSTRIDE + row];
                    u[x].l = s[G::GROUP * G::OSTRIDE + G::GROUP + row];
                    u[x].o = *reinterpret_cast<const float4*>(s + row * G::OSTRIDE + c);
                }
                acc.add(u);
            }
            if (whole) {
                acc.finish(p, q.b, head0 + row, c, D);
            } else {
                __stcg(reinterpret_cast<float4*>(mine + 2 * G::GROUP + row * D + c), acc.o);
                if (c == 0) {
                    __stcg(mine + row, acc.m);
                    __stcg(mine + G::GROUP + row, acc.l);
                }
            }
        }
        if (!whole) open[nopen++] = q;
    }
    if (nopen == 0) return;

    // ---- groups shared with other CTAs: the one that arrives last joins their
    // partial results (the count releases what the whole CTA has stored)
    __syncthreads();
    if (tid < nopen) {
        const Range& o = tid == 0 ? open[0] : open[1];
        const uint32_t c0 = cut_at.owner(o.begin), n = cut_at.owner(o.begin + o.tiles - 1) - c0 + 1;
        uint32_t* a = p.arrived + size_t(o.b) * groups + o.g;
        const bool last = atom_add_acq_rel_u32(a, 1u) == n - 1;
        if (last) *a = 0u;
        small[4 * tid] = last ? n : 0u;
        small[4 * tid + 1] = c0;
        small[4 * tid + 2] = cut_at.start(c0) >= o.begin ? 0u : 1u;
    }
    __syncthreads();
    for (int i = 0; i < nopen; ++i)
        if (small[4 * i])
            join_group<D, R>(p, i == 0 ? open[0] : open[1], small[4 * i + 1], int(small[4 * i]), small[4 * i + 2], tails);
}

template <int D, int R>
cudaError_t launch_attn(AttnParams& p, int grid, cudaStream_t st) {
    using G = Geo<D, R>;
    p.chunks = (p.per_kv + G::GROUP - 1) / G::GROUP;
    p.groups = p.chunks * p.Hkv;
    mk_paged_attention_kernel<D, R><<<grid, G::THREADS, G::SMEM, st>>>(p);
    return cudaGetLastError();
}

// Groups of up to 16 query heads per sequence, 0 for sizes outside the limits.
int64_t attn_groups(int B, int Hq, int Hkv) {
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return 0;
    return int64_t(Hkv) * ((Hq / Hkv + ROWS - 1) / ROWS);
}

template <int D, int R>
cudaError_t attn_smem() {
    return cudaFuncSetAttribute(mk_paged_attention_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Geo<D, R>::SMEM);
}

}  // namespace

cudaError_t attn_kernel_attributes() {
    cudaError_t e;
    if ((e = attn_smem<64, 1>()) != cudaSuccess || (e = attn_smem<64, 2>()) != cudaSuccess ||
        (e = attn_smem<128, 1>()) != cudaSuccess || (e = attn_smem<128, 2>()) != cudaSuccess)
        return e;
    return attn_smem<256, 1>();
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_paged_attention_workspace_size(int B, int Hq, int Hkv) {
    const int64_t g = attn_groups(B, Hq, Hkv);
    if (g == 0 || B > ATTN_MAX_B) return 0;
    return ATTN_SLOTS_BYTES + ws_align(size_t(B) * size_t(g) * sizeof(uint32_t));
}

extern "C" mk_status_t mk_paged_attention(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                          int64_t page_stride, int64_t token_stride, int64_t head_stride,
                                          const int32_t* block_table, const int32_t* seq_lens, int B, int Hq, int Hkv,
                                          int D, int page_size, int max_pages, int num_pages, float scale, void* out,
                                          float* lse, void* stream, void* workspace, size_t ws_bytes) {
    if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || page_size < 1 || max_pages < 0 || num_pages < 0)
        return MK_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return MK_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return MK_ERR_INVALID_ARG;
    const int64_t groups = attn_groups(B, Hq, Hkv);
    const int64_t cap = int64_t(max_pages) * page_size;
    if (B > ATTN_MAX_B || cap > (int64_t(1) << 31) - 32) return MK_ERR_UNSUPPORTED;
    // positions in the order of tiles are 32-bit
    const int64_t tiles = int64_t(B) * positions_of(int(cap), D == 64 ? Geo<64, 1>::KEYS : Geo<128, 1>::KEYS);
    if (tiles >= int64_t(1) << 31 || tiles * groups >= int64_t(1) << 31) return MK_ERR_UNSUPPORTED;
    if (B > 0) {
        if (!q || !seq_lens || !out) return MK_ERR_INVALID_ARG;
        if (cap > 0 && (!k_cache || !v_cache || !block_table || num_pages < 1)) return MK_ERR_INVALID_ARG;
        if (!host_aligned(q, 4) || !host_aligned(out, 8) || !host_aligned(k_cache, 16) || !host_aligned(v_cache, 16) ||
            !host_aligned(block_table, 4) || !host_aligned(seq_lens, 4) || !host_aligned(lse, 4))
            return MK_ERR_INVALID_ARG;
        if (B > 1 && (q_stride < int64_t(Hq) * D || q_stride % 2 != 0)) return MK_ERR_INVALID_ARG;
        // rows are copied in 16-byte pieces; the stride of a dimension of one is never used
        const int64_t used[3] = {num_pages > 1 ? page_stride : 0, page_size > 1 ? token_stride : 0,
                                 Hkv > 1 ? head_stride : 0};
        for (const int64_t v : used)
            if (v < 0 || v % 8 != 0) return MK_ERR_INVALID_ARG;
    }
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    mk_status_t s = host_device(&dev, &sms, &err);
    if (s != MK_OK) return s;
    if (B == 0) return MK_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t need = mk_paged_attention_workspace_size(B, Hq, Hkv);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Workspace cached;  // held until the launch below
    if (ws) {
        if (ws_bytes < need || !host_aligned(ws, 256)) return MK_ERR_WORKSPACE;
    } else {
        if ((s = cached.get(WS_ATTN, dev, st, need, need)) != MK_OK) return s;
        ws = cached.data();
    }
    AttnParams p{};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k_cache);
    p.v = static_cast<const __nv_bfloat16*>(v_cache);
    p.table = block_table;
    p.lens = seq_lens;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.slots = reinterpret_cast<float*>(ws);
    p.arrived = reinterpret_cast<uint32_t*>(ws + ATTN_SLOTS_BYTES);
    p.err = err;
    p.q_stride = q_stride;
    p.page_stride = page_stride;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.per_kv = Hq / Hkv;
    p.scale2 = scale * LOG2E;
    const int grid = std::min(sms, ATTN_MAX_CTAS);
    // Groups of 32 heads, two warps on a tile, where groups of 16 would pass over the
    // keys an even number of times and there is a group of 32 per CTA: with that many
    // the passes over a group's keys follow one another on the same SM, and the later
    // ones find them in L2 no more (32 sequences of 4096 keys, 8 key-value heads, 24
    // query heads each: 136 us, with groups of 16 170).  With fewer groups the passes
    // run side by side, and groups of 16 have more ranges (one sequence of 8191 keys,
    // 32 heads: 27 us, with groups of 16 22); with an odd number the second warp of the
    // last group has nothing to do (16 sequences of 30000, 48 heads: 123 and 116).
    const int passes = (p.per_kv + ROWS - 1) / ROWS;
    const bool wide = passes % 2 == 0 && int64_t(B) * Hkv * (passes / 2) >= grid;
    const cudaError_t e = D == 256          ? launch_attn<256, 1>(p, grid, st)
                          : D == 128 && wide ? launch_attn<128, 2>(p, grid, st)
                          : D == 128         ? launch_attn<128, 1>(p, grid, st)
                          : wide             ? launch_attn<64, 2>(p, grid, st)
                                             : launch_attn<64, 1>(p, grid, st);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
