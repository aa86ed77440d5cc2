// mk_attn_split.cuh -- what the attention kernels over paged caches share: the
// cut of all sequences' keys into equal ranges, one per warp (or pair of warps),
// and the way their partial results come together.
//
// P, a kernel's parameters, has: lens, table, B, Hq, per_kv (query heads per
// key-value head), chunks (groups of query heads per key-value head), groups
// (per sequence), max_pages, page_size, out, lse, slots (two partial results per
// CTA), arrived (a counter per sequence and group, zero between calls), err, and
// value_factor(kv), what the output of a key-value head is multiplied by.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mk_common.h"
#include "mk_host.h"
#include "mk_ptx.cuh"

namespace mk {
namespace {

// A group counts as this many tiles more than it has: its queries, its first
// tile's latency and its result cost about that, and short groups would
// otherwise gather in a few warps.
constexpr uint32_t EXTRA = 3;
constexpr int ATTN_MAX_B = 4096;  // sequences (their tile counts sit in shared memory)
constexpr int ATTN_MAX_CTAS = 160;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// Floats of a partial result: maxima and sums of up to 32 heads of 128 columns, or
// 16 of 256, and their weighted sums of values.  Fixed, so the counters never move.
constexpr int ATTN_SLOT_FLOATS = 64 + 32 * 128;
constexpr size_t ATTN_SLOTS_BYTES = size_t(2) * ATTN_MAX_CTAS * ATTN_SLOT_FLOATS * 4;

__device__ __forceinline__ void attn_error(DevError* e, uint32_t site, uint32_t info) {
    if (atomicCAS(&e->code, 0u, uint32_t(ERR_FAULT)) == 0u) {
        e->site = site;
        e->cta = blockIdx.x;
        e->info = info;
    }
}

// 16 bytes global -> shared; zeros when !ok (the source is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// Tiles [t0, t1) of group g of sequence b.  In the order of positions that is
// cut into ranges, EXTRA positions stand before a group's first tile.
struct Range {
    int b, g;
    uint32_t t0, t1;
    uint32_t begin;  // position of the group's first tile
    uint32_t tiles;  // tiles of the group
};
__host__ __device__ inline uint32_t positions_of(int len, int keys) {
    return len > 0 ? (uint32_t(len) + uint32_t(keys) - 1) / uint32_t(keys) + EXTRA : 0u;
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

template <typename P>
__device__ __forceinline__ int length_of(const P& p, int b) {
    const int64_t cap = int64_t(p.max_pages) * p.page_size;
    const int n = __ldg(p.lens + b);
    return n < 0 ? 0 : n > cap ? int(cap) : n;
}

// Positions of one group of each sequence, summed over the sequences before it,
// into prefix[0 .. B], by a whole CTA; sequences without keys get zeros and -inf.
template <int D, int KEYS, int THREADS, typename P>
__device__ __forceinline__ void count_positions(const P& p, uint32_t* prefix, uint32_t* small) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t cap = int64_t(p.max_pages) * p.page_size;
    {
        const int per = (p.B + THREADS - 1) / THREADS;
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        uint32_t mine = 0;
        for (int b = b0; b < b1; ++b) {
            const int n = __ldg(p.lens + b);
            if ((n < 0 || n > cap) && blockIdx.x == 0) attn_error(p.err, SITE_SEQ_LEN, uint32_t(n));
            mine += positions_of(length_of(p, b), KEYS);
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
            base += positions_of(length_of(p, b), KEYS);
        }
        if (b1 == p.B && b0 < b1) prefix[p.B] = base;
        __syncthreads();
    }
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (prefix[b + 1] != prefix[b]) continue;
        uint2* o = reinterpret_cast<uint2*>(p.out + int64_t(b) * p.Hq * D);
        for (int i = tid; i < p.Hq * D / 4; i += THREADS) o[i] = make_uint2(0u, 0u);
        if (p.lse)
            for (int i = tid; i < p.Hq; i += THREADS) p.lse[int64_t(b) * p.Hq + i] = -INFINITY;
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
    template <typename P>
    __device__ void finish(const P& p, int b, int head, int c, int D) const {
        const int64_t at = int64_t(b) * p.Hq + head;
        const float inv = l == 0.f ? 0.f : p.value_factor(head / p.per_kv) / l;
        *reinterpret_cast<uint2*>(p.out + at * D + c) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (p.lse && c == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
};

// The result of a group from the partial results of CTAs [c0, c0 + n), by a
// whole CTA.  A thread takes four columns of one head and, where there are more threads than
// that, every parts-th piece; the parts are joined in shared memory.
template <int D, int GROUP, int THREADS, typename P>
__device__ void join_group(const P& p, const Range& r, uint32_t c0, int n, uint32_t which0, float* smem_f) {
    const int tid = threadIdx.x;
    const int kv = r.g / p.chunks, head0 = kv * p.per_kv + (r.g % p.chunks) * GROUP;
    const int heads = min(GROUP, (kv + 1) * p.per_kv - head0);
    const int items = heads * (D / 4), parts = min(n, max(1, THREADS / items));
    Part* red = reinterpret_cast<Part*>(smem_f);
    // the first CTA's piece may lie in its second slot; the others' ranges start in the group
    const float* first = p.slots + size_t(2 * c0 + which0) * ATTN_SLOT_FLOATS;
    const float* other = p.slots + size_t(2 * c0) * ATTN_SLOT_FLOATS;
    for (int i0 = 0; i0 < items; i0 += THREADS) {
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
                    if (at < n) u[x].load(at == 0 ? first : other + size_t(2 * at) * ATTN_SLOT_FLOATS, GROUP, row, c, D);
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

// What the CTA's ranges have of groups that none of them holds whole: joined in
// shared memory, and where other CTAs hold parts of them too, by the CTA that is
// done last, in the order of the keys.  pieces[2 i] and [2 i + 1] are range i's first
// and last group (tiles 0: none), in shared memory; `firsts` and `tails` hold the
// ranges' results, each GROUP rows of D + 8 floats, GROUP maxima and GROUP sums.
// Called after every warp has written its results; the groups that `cut_at`'s CTAs
// share arrive at p.arrived.
template <int D, int GROUP, int RANGES, int THREADS, typename P>
__device__ __forceinline__ void join_ranges(const P& p, const Range* pieces, float* tails, const float* firsts, uint32_t* small,
                                            const Cut& cut_at, uint32_t start, uint32_t end) {
    constexpr int OSTRIDE = D + 8, PART = GROUP * OSTRIDE + 2 * GROUP;
    static_assert(RANGES <= 16, "a bit for each piece");
    const int tid = threadIdx.x;
    const uint32_t groups = uint32_t(p.groups);
    __syncthreads();
    // Every warp sorts the pieces out for itself: those of a group follow one another.
    const int lane = tid & 31;
    const Range mine_piece = pieces[min(lane, 2 * RANGES - 1)];
    const bool on = lane < 2 * RANGES && mine_piece.tiles != 0;
    const uint32_t lower = (1u << lane) - 1u, all = __ballot_sync(0xffffffffu, on);
    const uint32_t begin_before = __shfl_sync(0xffffffffu, mine_piece.begin, 31 - __clz(int((all & lower) | 1u)));
    const uint32_t firsts_of = __ballot_sync(0xffffffffu, on && ((all & lower) == 0 || begin_before != mine_piece.begin));
    // groups shared with other CTAs: the first and the last one's
    uint32_t opens = __ballot_sync(0xffffffffu, (firsts_of >> lane & 1u) && !(mine_piece.begin >= start && mine_piece.begin + mine_piece.tiles <= end));
    const int nopen = __popc(opens);
    // four columns of a head each; a warp's are of one group
    const int items = (min(GROUP, p.per_kv) * (D / 4) + 31) & ~31;
    uint32_t groups_left = firsts_of;
    for (int item = tid; groups_left; item += THREADS) {
        for (; groups_left && item >= items; item -= items) groups_left &= groups_left - 1u;
        if (!groups_left) break;
        const uint32_t later = groups_left & (groups_left - 1u);
        const uint32_t same = all & ~((groups_left & (0u - groups_left)) - 1u) & (later ? (later & (0u - later)) - 1u : 0xffffffffu);
        const int row = item / (D / 4), c = (item % (D / 4)) * 4;
        const Range q = pieces[__ffs(int(same)) - 1];
        const int kv = q.g / p.chunks, head0 = kv * p.per_kv + (q.g % p.chunks) * GROUP;
        if (row >= min(GROUP, (kv + 1) * p.per_kv - head0)) continue;
        Part acc;
        for (uint32_t rest = same; rest;) {
            constexpr int BATCH = 4;
            Part u[BATCH];
#pragma unroll
            for (int x = 0; x < BATCH; ++x) {
                if (rest == 0) continue;
                const int i = __ffs(int(rest)) - 1, w = i >> 1;
                rest &= rest - 1;
                const float* s = (i & 1 ? tails : firsts) + w * PART;
                u[x].m = s[GROUP * OSTRIDE + row];
                u[x].l = s[GROUP * OSTRIDE + GROUP + row];
                u[x].o = *reinterpret_cast<const float4*>(s + row * OSTRIDE + c);
            }
            acc.add(u);
        }
        if (q.begin >= start && q.begin + q.tiles <= end) {
            acc.finish(p, q.b, head0 + row, c, D);
        } else {
            // a CTA's first shared group takes its first slot, its last one the second
            float* mine = p.slots + size_t(2 * blockIdx.x + (start >= q.begin ? 0 : 1)) * ATTN_SLOT_FLOATS;
            __stcg(reinterpret_cast<float4*>(mine + 2 * GROUP + row * D + c), acc.o);
            if (c == 0) {
                __stcg(mine + row, acc.m);
                __stcg(mine + GROUP + row, acc.l);
            }
        }
    }
    if (nopen == 0) return;

    // ---- groups shared with other CTAs: the one that arrives last joins their
    // partial results (the count releases what the whole CTA has stored)
    __syncthreads();
    if (tid < nopen) {
        const Range o = pieces[__ffs(int(tid == 0 ? opens : opens & (opens - 1u))) - 1];
        const uint32_t c0 = cut_at.owner(o.begin), n = cut_at.owner(o.begin + o.tiles - 1) - c0 + 1;
        uint32_t* a = p.arrived + size_t(o.b) * groups + o.g;
        const bool last = atom_add_acq_rel_u32(a, 1u) == n - 1;
        if (last) *a = 0u;
        small[4 * tid] = last ? n : 0u;
        small[4 * tid + 1] = c0;
        small[4 * tid + 2] = cut_at.start(c0) >= o.begin ? 0u : 1u;
    }
    __syncthreads();
    for (int i = 0; i < nopen; ++i, opens &= opens - 1u)
        if (small[4 * i])
            join_group<D, GROUP, THREADS>(p, pieces[__ffs(int(opens)) - 1], small[4 * i + 1], int(small[4 * i]), small[4 * i + 2],
                                          tails);
}

}  // namespace
}  // namespace mk
