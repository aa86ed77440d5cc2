// mk_pages.cu -- pages of a key-value cache: copied, shared between sequences,
// given back, given out for new tokens, and moved together.
//
// The state of a pool stays on the device: refs[p] counts the rows of the block
// table that hold page p (0: free), row s of the table the pages of sequence s,
// ceil(lens[s] / page_size) of them.  Everything is decided by whole numbers and
// the lowest free pages are given out first, in the order of the call's list, so
// equal states give equal results.  A call whose list is wrong (a sequence
// outside the table or named twice, too few free pages) changes nothing and is
// reported.
//
// The lists are short, so the latency of dependent loads and of the launches
// bounds all but the moved bytes, which go at the rate of a copy: units of 32 KiB,
// one per CTA at a time, 128 bytes in flight per thread.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "mk.h"
#include "mk_common.h"
#include "mk_fp4.cuh"
#include "mk_host.h"

namespace mk {
namespace {

constexpr int MAX_LIST = 4096;         // sequences of a call
constexpr int MAX_ROWS = 65536;        // rows of a block table
constexpr int MAX_PAGES = 1 << 30;
constexpr int MAX_CACHES = 128;        // buffers of one copying launch (its parameters)
constexpr int COPY_THREADS = 256;
constexpr int COPY_DEEP = 8;           // pieces in flight per thread
constexpr int PLAN_THREADS = 1024;

// Buffers whose pages move together.
struct Buffers {
    uint8_t* base[MAX_CACHES];
    int64_t stride[MAX_CACHES];        // bytes between pages
    uint32_t pieces[MAX_CACHES];       // vectors per page
    uint32_t first[MAX_CACHES + 1];    // units of a page before this buffer's
    uint8_t log[MAX_CACHES];           // log2 of the vector's bytes
    int n;
};

template <typename V>
__device__ __forceinline__ void copy_unit(V* dst, const V* src, uint32_t at, uint32_t n) {
    V v[COPY_DEEP];
#pragma unroll
    for (int i = 0; i < COPY_DEEP; ++i) {
        const uint32_t x = at + i * COPY_THREADS + threadIdx.x;
        if (x < n) v[i] = __ldcs(src + x);
    }
#pragma unroll
    for (int i = 0; i < COPY_DEEP; ++i) {
        const uint32_t x = at + i * COPY_THREADS + threadIdx.x;
        if (x < n) __stcs(dst + x, v[i]);
    }
}

// Pages src[i] to dst[i] for i < moves, in every buffer.
__device__ __forceinline__ void move_pages(const Buffers& b, const int32_t* src, const int32_t* dst, int moves, int num_pages,
                                           DevError* err) {
    const uint32_t units = b.first[b.n];
    for (int64_t u = blockIdx.x; u < int64_t(moves) * units; u += gridDim.x) {
        const int i = u <= UINT32_MAX ? int(uint32_t(u) / units) : int(u / units);
        const uint32_t in = uint32_t(u - int64_t(i) * units);
        int lo = 0, hi = b.n;  // the last buffer with first <= in
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (b.first[mid] <= in) lo = mid;
            else hi = mid;
        }
        const int from = src[i], to = dst[i];  // (not by the read-only path: the kernel before may have written them)
        if (from < 0 || from >= num_pages || to < 0 || to >= num_pages) {
            if (threadIdx.x == 0) cache_error(err, ERR_FAULT, SITE_PAGE_INDEX, uint32_t(from < 0 || from >= num_pages ? from : to));
            continue;
        }
        const uint32_t at = (in - b.first[lo]) * (COPY_THREADS * COPY_DEEP), n = b.pieces[lo];
        const uint8_t* s = b.base[lo] + from * b.stride[lo];
        uint8_t* d = b.base[lo] + to * b.stride[lo];
        if (b.log[lo] == 4) copy_unit(reinterpret_cast<uint4*>(d), reinterpret_cast<const uint4*>(s), at, n);
        else if (b.log[lo] == 2) copy_unit(reinterpret_cast<uint32_t*>(d), reinterpret_cast<const uint32_t*>(s), at, n);
        else copy_unit(d, s, at, n);
    }
}

__global__ void __launch_bounds__(COPY_THREADS) mk_copy_pages_kernel(const __grid_constant__ Buffers b, const int32_t* src,
                                                                     const int32_t* dst, int moves, int num_pages, DevError* err) {
    move_pages(b, src, dst, moves, num_pages, err);
}

// A kernel that was launched to start beside the one before it waits here until that
// one is done and its results are seen.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct Pool {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    DevError* err;
    int rows, max_pages, num_pages, page_size;

    __device__ int pages_of(int len) const {
        return len <= 0 ? 0 : int(min(int64_t(max_pages), (int64_t(len) + page_size - 1) / page_size));
    }
    __device__ bool holds(int page) const { return page >= 0 && page < num_pages; }
};

// Whether the list's sequences all lie in the table and none is named twice; by
// a whole CTA.  `seen` holds a bit per row.
__device__ bool list_is_good(const Pool& p, const int32_t* list, int n, uint32_t* seen, int* bad) {
    for (int i = threadIdx.x; i < (p.rows + 31) / 32; i += blockDim.x) seen[i] = 0;
    if (threadIdx.x == 0) *bad = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int s = __ldg(list + i);
        if (s < 0 || s >= p.rows || (atomicOr(seen + (s >> 5), 1u << (s & 31)) >> (s & 31) & 1u)) atomicMin(bad, i);
    }
    __syncthreads();
    const int which = *bad;
    __syncthreads();  // the caller may use `bad` on
    if (which == INT_MAX) return true;
    if (threadIdx.x == 0 && blockIdx.x == 0) cache_error(p.err, ERR_FAULT, SITE_SEQUENCE, uint32_t(which));
    return false;
}

// ---- fork: the children give their pages back and hold their parents'

__device__ __forceinline__ void count_page(const Pool& p, int page, int by) {
    if (p.holds(page)) atomicAdd(p.refs + page, by);
    else cache_error(p.err, ERR_FAULT, SITE_PAGE_INDEX, uint32_t(page));
}
__device__ bool fork_is_good(const Pool& p, const int32_t* parent, const int32_t* child, int n, uint32_t* seen, int* bad) {
    if (!list_is_good(p, child, n, seen, bad)) return false;
    for (int j = threadIdx.x; j < n; j += blockDim.x) {  // a parent may be named any number of times
        const int s = __ldg(parent + j);
        if (s < 0 || s >= p.rows) atomicMin(bad, j);
    }
    __syncthreads();
    if (*bad == INT_MAX) return true;
    if (threadIdx.x == 0 && blockIdx.x == 0) cache_error(p.err, ERR_FAULT, SITE_SEQUENCE, uint32_t(*bad));
    return false;
}
// First the counts, a CTA per pair, and the lengths as they were; lens_before[i]: -1 when
// the call is refused.
__global__ void __launch_bounds__(256) mk_fork_count_kernel(Pool p, const int32_t* parent, const int32_t* child, int n,
                                                            int32_t* lens_before) {
    __shared__ uint32_t seen[MAX_ROWS / 32];
    __shared__ int bad;
    const int i = blockIdx.x;
    if (!fork_is_good(p, parent, child, n, seen, &bad)) {
        if (threadIdx.x == 0) lens_before[i] = -1;
        return;
    }
    const int from = __ldg(parent + i), to = __ldg(child + i), len = p.lens[from];
    const int32_t *theirs = p.table + int64_t(from) * p.max_pages, *own = p.table + int64_t(to) * p.max_pages;
    const int np = p.pages_of(len), no = p.pages_of(p.lens[to]);
    for (int j = threadIdx.x; j < max(np, no); j += 256) {
        if (j < np) count_page(p, theirs[j], 1);
        if (j < no) count_page(p, own[j], -1);
    }
    if (threadIdx.x == 0) lens_before[i] = max(len, 0);
}
// Then the rows.  A child may be another's parent, so a CTA takes all pairs' entries of
// some columns into registers before it writes any of them: rows of any length need no
// memory beside the table (224 pairs of 125 pages 7.0 us; with the parents' rows copied
// aside by the counting launch 6.0, but 64 of 8192 pages 21.7 for 20.4).  LIST: pairs at
// most.  COLS: a sector of a row, or half of one where a CTA has many pairs.
template <int LIST, int THREADS, int COLS>
__global__ void __launch_bounds__(THREADS) mk_fork_rows_kernel(Pool p, const int32_t* parent, const int32_t* child, int n,
                                                               const int32_t* lens_before) {
    constexpr int DEEP = LIST * COLS / THREADS, AT_ONCE = THREADS / COLS;
    static_assert(MAX_ROWS <= 65536, "two rows in a word");
    __shared__ uint32_t pairs[LIST];
    __shared__ int held[LIST];
    __shared__ int most;
    const int tid = threadIdx.x;
    for (int i = tid; i < n; i += THREADS) pairs[i] = uint32_t(__ldg(parent + i)) << 16 | (uint32_t(__ldg(child + i)) & 0xffffu);
    if (tid == 0) most = 0;
    wait_for_previous();
    __syncthreads();
    int longest = 0;
    for (int i = tid; i < n; i += THREADS) {
        const int len = lens_before[i];
        held[i] = p.pages_of(len);
        longest = max(longest, held[i]);  // stays 0 when the call is refused
        if (blockIdx.x == 0 && len >= 0) p.lens[pairs[i] & 0xffffu] = len;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (tid % 32 == 0 && longest > 0) atomicMax(&most, longest);
    __syncthreads();
    for (uint32_t c0 = blockIdx.x * COLS; c0 < uint32_t(most); c0 += gridDim.x * COLS) {
        const uint32_t col = c0 + tid % COLS;
        int v[DEEP];
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
            const int i = k * AT_ONCE + tid / COLS;
            if (i < n && col < uint32_t(held[i])) v[k] = p.table[int64_t(pairs[i] >> 16) * p.max_pages + col];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
            const int i = k * AT_ONCE + tid / COLS;
            if (i < n && col < uint32_t(held[i])) p.table[int64_t(pairs[i] & 0xffffu) * p.max_pages + col] = v[k];
        }
    }
}
// All of it by one CTA, a warp per pair and 128 columns at a time: for a few sequences one
// launch less on the host (32 pairs of 125 pages 5.4 us, 33 of them by the two above 6.1;
// long rows want more CTAs, 32 of 4096 pages 69, 64 of 8192 20).
constexpr int FORK_FEW = PLAN_THREADS / 32;
__global__ void __launch_bounds__(PLAN_THREADS) mk_fork_few_kernel(Pool p, const int32_t* parent, const int32_t* child, int n) {
    __shared__ uint32_t seen[MAX_ROWS / 32];
    __shared__ int bad, most;
    if (threadIdx.x == 0) most = 0;
    if (!fork_is_good(p, parent, child, n, seen, &bad)) return;
    const int i = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int from = 0, to = 0, len = 0, np = 0, no = 0;
    if (i < n) {
        from = __ldg(parent + i);
        to = __ldg(child + i);
        len = max(p.lens[from], 0);
        np = p.pages_of(len);
        no = p.pages_of(p.lens[to]);
        if (lane == 0) atomicMax(&most, max(np, no));
    }
    __syncthreads();  // every length has been read
    if (i < n && lane == 0) p.lens[to] = len;
    const int32_t* theirs = p.table + int64_t(from) * p.max_pages;
    int32_t* own = p.table + int64_t(to) * p.max_pages;
    constexpr int DEEP = 4;
    for (int64_t c0 = 0; c0 < most; c0 += 32 * DEEP) {
        int v[DEEP];
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
            const int64_t j = c0 + k * 32 + lane;
            if (j < np) count_page(p, v[k] = theirs[j], 1);
            if (j < no) count_page(p, own[j], -1);
        }
        __syncthreads();  // every pair's entries of these columns have been read
#pragma unroll
        for (int k = 0; k < DEEP; ++k) {
            const int64_t j = c0 + k * 32 + lane;
            if (j < np) own[j] = v[k];
        }
    }
}

// ---- free

__global__ void __launch_bounds__(256) mk_free_kernel(Pool p, const int32_t* seqs, int n) {
    __shared__ uint32_t seen[MAX_ROWS / 32];
    __shared__ int bad, len;
    if (!list_is_good(p, seqs, n, seen, &bad)) return;
    const int s = __ldg(seqs + blockIdx.x);
    if (threadIdx.x == 0) {
        len = p.lens[s];
        p.lens[s] = 0;
    }
    __syncthreads();
    const int np = p.pages_of(len);
    for (int j = threadIdx.x; j < np; j += blockDim.x) {
        const int page = p.table[int64_t(s) * p.max_pages + j];
        if (p.holds(page)) atomicSub(p.refs + page, 1);
        else cache_error(p.err, ERR_FAULT, SITE_PAGE_INDEX, uint32_t(page));
    }
}

// ---- extend: room for new tokens

// Sums over a CTA: the sum of what the threads before this one have; *total of all.
__device__ __forceinline__ int scan(int mine, int* part, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += o;
    }
    __syncthreads();  // the buffer is free
    if (lane == 31) part[warp] = run;
    __syncthreads();
    if (warp == 0) {
        int v = lane < warps ? part[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += o;
        }
        part[lane] = v;
    }
    __syncthreads();
    *total = part[warps - 1];
    return run - mine + (warp ? part[warp - 1] : 0);
}

// What the second kernel of an extension finds in the workspace.
struct Extension {
    int32_t ok, moves;
};

// Reports what entry i of an extension's list is refused for.
__device__ void extend_error(const Pool& p, const int32_t* seqs, const int32_t* count, int most, int i) {
    const int s = __ldg(seqs + i), more = __ldg(count + i), len = p.lens[s];
    if (more < 0 || more > most || len < 0) {
        cache_error(p.err, ERR_FAULT, SITE_TOKEN_COUNT, uint32_t(i));
        return;
    }
    const int64_t pages = (int64_t(len) + more + p.page_size - 1) / p.page_size;
    if (pages > p.max_pages) cache_error(p.err, ERR_FAULT, SITE_POOL_FULL, uint32_t(pages - p.max_pages));
    else cache_error(p.err, ERR_FAULT, SITE_PAGE_INDEX, uint32_t(p.table[int64_t(s) * p.max_pages + len / p.page_size]));
}

// Decides everything, by one CTA: which shared pages are copied (src, dst), which
// pages each sequence gets, their lengths.  `fresh` has room for num_pages.
__global__ void __launch_bounds__(PLAN_THREADS) mk_extend_plan_kernel(Pool p, const int32_t* seqs, const int32_t* count, int n, int most,
                                                                      Extension* head, int32_t* src, int32_t* dst, int32_t* fresh) {
    __shared__ uint32_t seen[MAX_ROWS / 32];
    __shared__ int last[MAX_LIST];    // the page that a sequence is in the middle of, or -1
    __shared__ int first[MAX_LIST];   // its place among the fresh pages
    __shared__ int part[32];
    __shared__ int bad;
    __shared__ unsigned long long wanted;  // pages, at most
    const int tid = threadIdx.x;
    if (tid == 0) wanted = 0;
    bool good = list_is_good(p, seqs, n, seen, &bad);
    if (good) {
        for (int i = tid; i < n; i += PLAN_THREADS) {
            const int s = __ldg(seqs + i), more = __ldg(count + i), len = p.lens[s];
            const int64_t cap = int64_t(p.max_pages) * p.page_size;
            if (more < 0 || more > most || len < 0 || len + int64_t(more) > cap) {
                atomicMin(&bad, i);
                continue;
            }
            int page = -1;
            if (more > 0 && len % p.page_size != 0) {
                page = p.table[int64_t(s) * p.max_pages + len / p.page_size];
                if (!p.holds(page)) atomicMin(&bad, i);
            }
            last[i] = page;
            // of all sequences they may pass 32 bits, in which they are counted below
            if (int64_t(n) * p.max_pages > INT_MAX)
                atomicAdd(&wanted, static_cast<unsigned long long>(p.pages_of(len + more) - p.pages_of(len)));
        }
        __syncthreads();
        good = bad == INT_MAX;
        if (!good && tid == 0) extend_error(p, seqs, count, most, bad);
    }
    // Whether a sequence copies the page that it is in the middle of: if others hold it
    // still when those before it in the list have left it (the last of them keeps it).
    const auto copies_page = [&](int i) {
        const int page = last[i];
        if (page < 0) return false;
        const int holders = p.refs[page];
        if (holders <= 1) return false;
        int before = 0;
        for (int j = 0; j < i; ++j) before += last[j] == page;
        return holders - before > 1;
    };
    if (good && wanted > static_cast<unsigned long long>(p.num_pages)) {
        good = false;
        for (int i = tid; i < n; i += PLAN_THREADS)
            if (copies_page(i)) atomicAdd(&wanted, 1ull);
        int mine = 0, free;
        for (int at = tid; at < p.num_pages; at += PLAN_THREADS) mine += p.refs[at] == 0;
        scan(mine, part, &free);
        if (tid == 0) cache_error(p.err, ERR_FAULT, SITE_POOL_FULL, uint32_t(min(wanted - free, static_cast<unsigned long long>(INT_MAX))));
    }
    if (!good) {
        if (tid == 0) *head = Extension{0, 0};
        return;
    }
    int need = 0, moved = 0;
    for (int i0 = 0; i0 < n; i0 += PLAN_THREADS) {
        const int i = i0 + tid;
        int mine = 0;
        bool copies = false;
        if (i < n) {
            copies = copies_page(i);
            const int s = __ldg(seqs + i), len = p.lens[s];
            mine = p.pages_of(len + __ldg(count + i)) - p.pages_of(len) + copies;
        }
        int total, moves;
        const int at = scan(mine, part, &total), m = scan(copies, part, &moves);
        if (i < n) {
            first[i] = need + at;
            if (copies) {
                src[moved + m] = last[i];
                dst[moved + m] = i;  // for now: whose
            }
        }
        need += total;
        moved += moves;
    }
    // the lowest free pages: a lane takes 32 neighbouring ones, which its warp reads together
    int found = 0;
    const int warp = tid >> 5, lane = tid & 31;
    for (int p0 = 0; p0 < p.num_pages && found < need; p0 += PLAN_THREADS * 32) {
        const int first_page = p0 + warp * 1024;
        uint32_t free = 0;
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += 8) {
            if (first_page + k0 * 32 >= p.num_pages) break;  // the same for the whole warp
            int r[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int at = first_page + (k0 + k) * 32 + lane;
                r[k] = at < p.num_pages ? p.refs[at] : 1;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t word = __ballot_sync(0xffffffffu, r[k] == 0);
                if (lane == k0 + k) free = word;
            }
        }
        int total;
        int to = found + scan(__popc(free), part, &total);
        for (; free && to < need; free &= free - 1) fresh[to++] = first_page + lane * 32 + __ffs(free) - 1;
        found += total;
    }
    if (found < need) {
        if (tid == 0) {
            cache_error(p.err, ERR_FAULT, SITE_POOL_FULL, uint32_t(need - found));
            *head = Extension{0, 0};
        }
        return;
    }
    __syncthreads();  // every page has been looked at, and fresh is whole
    for (int i = tid; i < need; i += PLAN_THREADS) p.refs[fresh[i]] = 1;
    // a copied page is the first of its sequence's
    for (int m = tid; m < moved; m += PLAN_THREADS) {
        const int i = dst[m], s = __ldg(seqs + i);
        atomicSub(p.refs + src[m], 1);
        const int to = fresh[first[i]];
        p.table[int64_t(s) * p.max_pages + p.lens[s] / p.page_size] = to;
        dst[m] = to;
        last[i] = -2;
    }
    __syncthreads();
    for (int i = warp; i < n; i += PLAN_THREADS / 32) {
        const int s = __ldg(seqs + i), len = p.lens[s], more = __ldg(count + i);
        const int have = p.pages_of(len), want = p.pages_of(len + more), from = first[i] + (last[i] == -2);
        __syncwarp();
        for (int j = have + lane; j < want; j += 32) p.table[int64_t(s) * p.max_pages + j] = fresh[from + j - have];
        if (lane == 0) p.lens[s] = len + more;
    }
    if (tid == 0) *head = Extension{1, moved};
}
// The copies, and the places of the new tokens.
__global__ void __launch_bounds__(COPY_THREADS) mk_extend_kernel(Pool p, const __grid_constant__ Buffers b, const int32_t* seqs,
                                                                 const int32_t* count, int n, int most, const Extension* head,
                                                                 const int32_t* src, const int32_t* dst, int64_t* slots) {
    wait_for_previous();
    const Extension e = *head;
    if (slots)
        for (int64_t x = int64_t(blockIdx.x) * COPY_THREADS + threadIdx.x; x < int64_t(n) * most; x += int64_t(gridDim.x) * COPY_THREADS) {
            const int i = int(x / most), j = int(x - int64_t(i) * most);
            int64_t slot = -1;
            if (e.ok && j < __ldg(count + i)) {
                const int s = __ldg(seqs + i), at = p.lens[s] - __ldg(count + i) + j, k = at / p.page_size;
                slot = int64_t(p.table[int64_t(s) * p.max_pages + k]) * p.page_size + (at - k * p.page_size);
            }
            slots[x] = slot;
        }
    if (e.ok && b.n > 0) move_pages(b, src, dst, e.moves, p.num_pages, p.err);
}
// The copies of the buffers beyond MAX_CACHES.
__global__ void __launch_bounds__(COPY_THREADS) mk_extend_more_kernel(Pool p, const __grid_constant__ Buffers b, const Extension* head,
                                                                      const int32_t* src, const int32_t* dst) {
    const Extension e = *head;
    if (e.ok) move_pages(b, src, dst, e.moves, p.num_pages, p.err);
}

// ---- compact: the pages in use become the first ones

// Of each part of the pool: how many of its pages are in use.
__global__ void __launch_bounds__(256) mk_compact_count_kernel(const int32_t* refs, int num_pages, int each, int32_t* counts) {
    __shared__ int part[32];
    int mine = 0;
    const int p0 = blockIdx.x * each, p1 = min(num_pages, p0 + each);
    for (int i = p0 + threadIdx.x; i < p1; i += 256) mine += __ldg(refs + i) > 0;
    int total;
    scan(mine, part, &total);
    if (threadIdx.x == 0) counts[blockIdx.x] = total;
}
// With `used` pages in use: the i-th free one below that takes the i-th used one
// above.  rank[page] of a page above: its i.
struct Compaction {
    int32_t used, moves;
};
__global__ void __launch_bounds__(256) mk_compact_plan_kernel(const int32_t* refs, int num_pages, int each, const int32_t* counts,
                                                              Compaction* head, int32_t* src, int32_t* dst, int32_t* rank) {
    __shared__ int part[32];
    wait_for_previous();
    const int tid = threadIdx.x, parts = gridDim.x;
    int used = 0, before = 0;
    for (int i = tid; i < parts; i += 256) {
        const int c = counts[i];
        used += c;
        before += i < int(blockIdx.x) ? c : 0;
    }
    int total, mine_before, below;
    scan(used, part, &total);
    scan(before, part, &mine_before);
    // pages in use below `total`: whole parts, and a part of one
    int some = 0;
    const int cut = total / each;
    for (int i = tid; i < cut; i += 256) some += counts[i];
    for (int i = cut * each + tid; i < total; i += 256) some += __ldg(refs + i) > 0;
    scan(some, part, &below);
    if (blockIdx.x == 0 && tid == 0) *head = Compaction{total, total - below};
    const int p0 = blockIdx.x * each, p1 = min(num_pages, p0 + each);
    int seen = mine_before;
    for (int i0 = p0; i0 < p1; i0 += 256) {
        const int i = i0 + tid;
        const bool on = i < p1 && __ldg(refs + i) > 0;
        int some_used;
        const int at = seen + scan(on, part, &some_used);  // pages in use before i
        if (i < p1) {
            if (i < total && !on) dst[i - at] = i;
            if (i >= total && on) {
                src[at - below] = i;
                rank[i] = at - below;
            }
        }
        seen += some_used;
    }
}
struct CompactOut {
    const int32_t* table;
    const int32_t* refs;
    int32_t* table_out;
    int32_t* refs_out;
};
__global__ void __launch_bounds__(COPY_THREADS) mk_compact_kernel(Pool p, CompactOut c, const __grid_constant__ Buffers b, const Compaction* head,
                                                                  const int32_t* src, const int32_t* dst, const int32_t* rank) {
    wait_for_previous();
    const Compaction e = *head;
    const int64_t t0 = int64_t(blockIdx.x) * COPY_THREADS + threadIdx.x, step = int64_t(gridDim.x) * COPY_THREADS;
    for (int64_t x = t0; x < int64_t(p.rows) * p.max_pages; x += step) {
        const int s = int(x / p.max_pages), j = int(x - int64_t(s) * p.max_pages);
        int page = c.table[x];
        if (j < p.pages_of(__ldg(p.lens + s))) {
            // a page that no row counts on is not moved: its entry stays
            if (!p.holds(page)) cache_error(p.err, ERR_FAULT, SITE_PAGE_INDEX, uint32_t(page));
            else if (page >= e.used && rank[page] >= 0 && rank[page] < e.moves && src[rank[page]] == page) page = dst[rank[page]];
        }
        if (c.table_out != c.table || page != c.table[x]) c.table_out[x] = page;
    }
    if (c.refs_out != c.refs)
        for (int64_t x = t0; x < p.num_pages; x += step) {
            const int r = c.refs[x];
            if (x < e.used ? r > 0 : r <= 0) c.refs_out[x] = r;
        }
    for (int64_t i = t0; i < e.moves; i += step) {  // alone with both
        const int r = c.refs[src[i]];
        c.refs_out[dst[i]] = r;
        c.refs_out[src[i]] = 0;
    }
    if (b.n > 0) move_pages(b, src, dst, e.moves, p.num_pages, p.err);
}
__global__ void __launch_bounds__(COPY_THREADS) mk_compact_more_kernel(Pool p, const __grid_constant__ Buffers b, const Compaction* head,
                                                                       const int32_t* src, const int32_t* dst) {
    move_pages(b, src, dst, head->moves, p.num_pages, p.err);
}

// ---- host

struct CacheList {
    void* const* base;
    const int64_t* stride;
    const int64_t* bytes;
    int n;
};

bool good_caches(const CacheList& c, int num_pages) {
    if (c.n < 0) return false;
    if (c.n > 0 && (!c.base || !c.stride || !c.bytes)) return false;
    for (int i = 0; i < c.n; ++i) {
        if (c.bytes[i] < 1 || c.bytes[i] > (int64_t(1) << 31)) return false;
        if (num_pages > 1 && c.stride[i] < c.bytes[i]) return false;
        if (num_pages > 0 && !c.base[i]) return false;
    }
    return true;
}

// Buffers [i0, i0 + MAX_CACHES) of the list.
Buffers some_buffers(const CacheList& c, int i0) {
    Buffers b{};
    b.n = std::max(0, std::min(MAX_CACHES, c.n - i0));
    for (int i = 0; i < b.n; ++i) {
        const int64_t bytes = c.bytes[i0 + i], stride = c.stride[i0 + i];
        const uintptr_t all = reinterpret_cast<uintptr_t>(c.base[i0 + i]) | uintptr_t(bytes) | uintptr_t(stride);
        const int log = all % 16 == 0 ? 4 : all % 4 == 0 ? 2 : 0;
        b.base[i] = static_cast<uint8_t*>(c.base[i0 + i]);
        b.stride[i] = stride;
        b.log[i] = uint8_t(log);
        b.pieces[i] = uint32_t(bytes >> log);
        constexpr uint32_t UNIT = COPY_THREADS * COPY_DEEP;
        b.first[i + 1] = b.first[i] + (b.pieces[i] + UNIT - 1) / UNIT;
    }
    return b;
}

int copy_grid(int sms) { return sms * 32; }

mk_status_t pool_arguments(const void* table, const void* lens, const void* refs, int rows, int max_pages, int num_pages,
                           int page_size, int n) {
    if (rows < 0 || max_pages < 0 || num_pages < 0 || page_size < 1 || n < 0) return MK_ERR_INVALID_ARG;
    if (rows > MAX_ROWS || n > MAX_LIST || num_pages > MAX_PAGES || int64_t(max_pages) * page_size > INT_MAX) return MK_ERR_UNSUPPORTED;
    if (rows > 0 && (!lens || (max_pages > 0 && !table))) return MK_ERR_INVALID_ARG;
    if (num_pages > 0 && !refs) return MK_ERR_INVALID_ARG;
    if (!host_aligned(table, 4) || !host_aligned(lens, 4) || !host_aligned(refs, 4)) return MK_ERR_INVALID_ARG;
    return MK_OK;
}
bool list_argument(const void* list, int n) { return n == 0 || (list && host_aligned(list, 4)); }

// The caller's workspace or the library's.
mk_status_t workspace_of(Workspace& cached, int dev, cudaStream_t st, void* workspace, size_t ws_bytes, size_t need, uint8_t** out) {
    if (workspace) {
        if (ws_bytes < need || !host_aligned(workspace, 256)) return MK_ERR_WORKSPACE;
        *out = static_cast<uint8_t*>(workspace);
        return MK_OK;
    }
    const mk_status_t s = cached.get(WS_PAGES, dev, st, need, 0);
    *out = cached.data();
    return s;
}
// Launches a kernel that begins with wait_for_previous(): its CTAs are set up while the
// one before it ends (1 us each).
template <typename... P, typename... A>
void launch_behind(void (*kernel)(P...), int grid, int threads, cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(unsigned(grid));
    c.blockDim = dim3(unsigned(threads));
    c.stream = st;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &a;
    c.numAttrs = 1;
    cudaLaunchKernelEx(&c, kernel, P(args)...);
}
mk_status_t launched() { return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA; }

constexpr size_t HEAD_BYTES = 256;

size_t fork_bytes(int n) { return ws_align(size_t(n) * 4); }
size_t extend_bytes(int num_pages, int n) { return HEAD_BYTES + 2 * ws_align(size_t(n) * 4) + ws_align(size_t(num_pages) * 4); }
size_t compact_bytes(int num_pages) { return HEAD_BYTES + ws_align(1024 * 4) + 3 * ws_align(size_t(num_pages) * 4); }

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" size_t mk_pages_workspace_size(int max_pages, int num_pages, int n) {
    if (max_pages < 0 || num_pages < 0 || n < 0 || n > MAX_LIST) return 0;
    return std::max({fork_bytes(n), extend_bytes(num_pages, n), compact_bytes(num_pages)});
}

extern "C" mk_status_t mk_copy_pages(void* const* caches, const int64_t* page_strides, const int64_t* page_bytes, int n_caches,
                                     int num_pages, const int32_t* src, const int32_t* dst, int n, void* stream) {
    const CacheList c{caches, page_strides, page_bytes, n_caches};
    if (num_pages < 0 || n < 0 || !good_caches(c, num_pages)) return MK_ERR_INVALID_ARG;
    if (!list_argument(src, n) || !list_argument(dst, n)) return MK_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    const mk_status_t s = host_device(&dev, &sms, &err);
    if (s != MK_OK) return s;
    if (n == 0) return MK_OK;
    for (int i = 0; i < n_caches; i += MAX_CACHES) {
        const Buffers b = some_buffers(c, i);
        const int64_t units = int64_t(n) * b.first[b.n];
        mk_copy_pages_kernel<<<int(std::min<int64_t>(units, copy_grid(sms))), COPY_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
            b, src, dst, n, num_pages, err);
    }
    return launched();
}

extern "C" mk_status_t mk_fork_sequences(int32_t* block_table, int32_t* seq_lens, int32_t* refs, int rows, int max_pages, int num_pages,
                                         int page_size, const int32_t* parent, const int32_t* child, int n, void* stream,
                                         void* workspace, size_t ws_bytes) {
    mk_status_t s = pool_arguments(block_table, seq_lens, refs, rows, max_pages, num_pages, page_size, n);
    if (s != MK_OK) return s;
    if (!list_argument(parent, n) || !list_argument(child, n)) return MK_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    if ((s = host_device(&dev, &sms, &err)) != MK_OK) return s;
    if (n == 0) return MK_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Pool p{block_table, seq_lens, refs, err, rows, max_pages, num_pages, page_size};
    Workspace cached;
    uint8_t* ws = nullptr;
    if (workspace || n > FORK_FEW)
        if ((s = workspace_of(cached, dev, st, workspace, ws_bytes, fork_bytes(n), &ws)) != MK_OK) return s;
    if (n <= FORK_FEW) {
        mk_fork_few_kernel<<<1, PLAN_THREADS, 0, st>>>(p, parent, child, n);
    } else {
        int32_t* lens_before = reinterpret_cast<int32_t*>(ws);
        mk_fork_count_kernel<<<n, 256, 0, st>>>(p, parent, child, n, lens_before);
        const auto rows_of = [&](auto kernel, int threads, int cols, int each) {  // `each` CTAs of an SM
            const int grid = std::max(1, std::min(sms * each, (max_pages - 1) / cols + 1));
            launch_behind(kernel, grid, threads, st, p, parent, child, n, lens_before);
        };
        if (n <= 256) rows_of(mk_fork_rows_kernel<256, 256, 8>, 256, 8, 8);
        else if (n <= 1024) rows_of(mk_fork_rows_kernel<1024, 256, 8>, 256, 8, 4);
        else rows_of(mk_fork_rows_kernel<MAX_LIST, PLAN_THREADS, 4>, PLAN_THREADS, 4, 1);
    }
    return launched();
}

extern "C" mk_status_t mk_free_sequences(const int32_t* block_table, int32_t* seq_lens, int32_t* refs, int rows, int max_pages,
                                         int num_pages, int page_size, const int32_t* seqs, int n, void* stream) {
    mk_status_t s = pool_arguments(block_table, seq_lens, refs, rows, max_pages, num_pages, page_size, n);
    if (s != MK_OK) return s;
    if (!list_argument(seqs, n)) return MK_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    if ((s = host_device(&dev, &sms, &err)) != MK_OK) return s;
    if (n == 0) return MK_OK;
    const Pool p{const_cast<int32_t*>(block_table), seq_lens, refs, err, rows, max_pages, num_pages, page_size};
    mk_free_kernel<<<n, 256, 0, static_cast<cudaStream_t>(stream)>>>(p, seqs, n);
    return launched();
}

extern "C" mk_status_t mk_extend_sequences(int32_t* block_table, int32_t* seq_lens, int32_t* refs, int rows, int max_pages,
                                           int num_pages, int page_size, const int32_t* seqs, const int32_t* count, int n, int most,
                                           int64_t* slots, void* const* caches, const int64_t* page_strides,
                                           const int64_t* page_bytes, int n_caches, void* stream, void* workspace, size_t ws_bytes) {
    mk_status_t s = pool_arguments(block_table, seq_lens, refs, rows, max_pages, num_pages, page_size, n);
    if (s != MK_OK) return s;
    const CacheList c{caches, page_strides, page_bytes, n_caches};
    if (most < 0 || !list_argument(seqs, n) || !list_argument(count, n) || !host_aligned(slots, 8) || !good_caches(c, num_pages))
        return MK_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    if ((s = host_device(&dev, &sms, &err)) != MK_OK) return s;
    if (n == 0) return MK_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    Workspace cached;
    uint8_t* ws = nullptr;
    if ((s = workspace_of(cached, dev, st, workspace, ws_bytes, extend_bytes(num_pages, n), &ws)) != MK_OK) return s;
    Extension* head = reinterpret_cast<Extension*>(ws);
    int32_t* src = reinterpret_cast<int32_t*>(ws + HEAD_BYTES);
    int32_t* dst = reinterpret_cast<int32_t*>(ws + HEAD_BYTES + ws_align(size_t(n) * 4));
    int32_t* fresh = reinterpret_cast<int32_t*>(ws + HEAD_BYTES + 2 * ws_align(size_t(n) * 4));
    const Pool p{block_table, seq_lens, refs, err, rows, max_pages, num_pages, page_size};
    mk_extend_plan_kernel<<<1, PLAN_THREADS, 0, st>>>(p, seqs, count, n, most, head, src, dst, fresh);
    for (int i = 0; i < std::max(1, n_caches); i += MAX_CACHES) {
        const Buffers b = some_buffers(c, i);
        const int64_t work = std::max<int64_t>(int64_t(n) * b.first[b.n], (int64_t(n) * most + COPY_THREADS - 1) / COPY_THREADS);
        const int grid = int(std::max<int64_t>(1, std::min<int64_t>(work, copy_grid(sms))));
        if (i == 0) launch_behind(mk_extend_kernel, grid, COPY_THREADS, st, p, b, seqs, count, n, most, head, src, dst, slots);
        else mk_extend_more_kernel<<<grid, COPY_THREADS, 0, st>>>(p, b, head, src, dst);
    }
    return launched();
}

extern "C" mk_status_t mk_compact_pages(const int32_t* block_table, const int32_t* seq_lens, const int32_t* refs, int rows,
                                        int max_pages, int num_pages, int page_size, int32_t* table_out, int32_t* refs_out,
                                        void* const* caches, const int64_t* page_strides, const int64_t* page_bytes, int n_caches,
                                        void* stream, void* workspace, size_t ws_bytes) {
    mk_status_t s = pool_arguments(block_table, seq_lens, refs, rows, max_pages, num_pages, page_size, 0);
    if (s != MK_OK) return s;
    const CacheList c{caches, page_strides, page_bytes, n_caches};
    if (!good_caches(c, num_pages) || (num_pages > 0 && !refs_out) || (rows > 0 && max_pages > 0 && !table_out) ||
        !host_aligned(table_out, 4) || !host_aligned(refs_out, 4))
        return MK_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    if ((s = host_device(&dev, &sms, &err)) != MK_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (num_pages == 0) {
        const size_t bytes = size_t(rows) * size_t(max_pages) * 4;
        if (table_out == block_table || bytes == 0) return MK_OK;
        return cudaMemcpyAsync(table_out, block_table, bytes, cudaMemcpyDeviceToDevice, st) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
    }
    Workspace cached;
    uint8_t* ws = nullptr;
    if ((s = workspace_of(cached, dev, st, workspace, ws_bytes, compact_bytes(num_pages), &ws)) != MK_OK) return s;
    Compaction* head = reinterpret_cast<Compaction*>(ws);
    int32_t* counts = reinterpret_cast<int32_t*>(ws + HEAD_BYTES);
    int32_t* src = counts + ws_align(1024 * 4) / 4;
    int32_t* dst = src + ws_align(size_t(num_pages) * 4) / 4;
    int32_t* rank = dst + ws_align(size_t(num_pages) * 4) / 4;
    // parts of at least 1024 pages, one per CTA of two small launches
    const int each = std::max(1024, (num_pages + std::min(sms, 1024) - 1) / std::min(sms, 1024));
    const int parts = (num_pages + each - 1) / each;
    const Pool p{nullptr, const_cast<int32_t*>(seq_lens), nullptr, err, rows, max_pages, num_pages, page_size};
    const CompactOut out{block_table, refs, table_out, refs_out};
    mk_compact_count_kernel<<<parts, 256, 0, st>>>(refs, num_pages, each, counts);
    launch_behind(mk_compact_plan_kernel, parts, 256, st, refs, num_pages, each, counts, head, src, dst, rank);
    for (int i = 0; i < std::max(1, n_caches); i += MAX_CACHES) {
        const Buffers b = some_buffers(c, i);
        if (i == 0) launch_behind(mk_compact_kernel, copy_grid(sms), COPY_THREADS, st, p, out, b, head, src, dst, rank);
        else mk_compact_more_kernel<<<copy_grid(sms), COPY_THREADS, 0, st>>>(p, b, head, src, dst);
    }
    return launched();
}
