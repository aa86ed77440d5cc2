// mk_ffn.cu -- mk_moe_ffn_decode: the whole gated expert layer for a few
// tokens in one persistent kernel.
//
//   experts of token t: the k largest logits; gates: softmax over them
//   h = silu(x . W1[e]) * (x . W3[e]),   out[t] = sum_j gate_j h . W2[e_j]
//
// For a few tokens the chosen experts' weights are all the traffic, each used
// for the few rows routed to its expert, so the kernel is a stream of
// weights: one step is 32 KiB of them, and the steps of all chosen experts in
// a row are cut into one equal range per CTA, first those of W1 and W3, then
// those of W2.  Every SM therefore reads the same number of bytes, whatever
// the routing.
//
// The products run on tcgen05 with the weights as the 128-row operand (their
// columns are its rows, M-major as they lie in memory, loaded by TMA) and the
// expert's rows of x or h as the N = 16..128 columns, gathered by TMA
// tile::gather4.  Roles of a CTA's warps: one loads weights and waits for
// nothing but free stages, so across the boundary between the two halves the
// stream goes on while h is still being completed; one gathers rows (and
// waits for an expert's h before its first use); one issues products; eight
// drain accumulators.
//
// A tile (128 columns of W1 and W3, or 256 of W2, over all of K) may be split
// over CTAs.  The pieces are fp32 sums in the workspace; for h the CTA that
// delivers the last piece of a tile adds them up in their order, applies
// SwiGLU and publishes the tile, and for the outputs the combine after the
// last barrier of the grid adds the pieces of each token's k rows in order.
// No result depends on which CTA was first.
//
// 16-bit weights: h is kept as the sum of two bf16 values (two products into
// one accumulator, 16 significant bits), since the tensor core has time to
// spare here and one rounding fewer reaches the output.  8-bit weights: a
// weight scale per 128 x 128 block and a scale of x and h per row and 128
// columns, so one step is one block of K; its products leave the tensor core
// after each step and are added up in fp32 registers with their scales.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk.h"
#include "mk_common.h"
#include "mk_host.h"
#include "mk_ptx.cuh"
#include "mk_wait.cuh"

namespace mk {
namespace {

constexpr int FFN_MAX_T = 128;
constexpr int FFN_MAX_ROWS = FFN_MAX_T * MAX_K;
constexpr int FFN_MAX_CTAS = 160;

// Warps: weight loads, products, eight draining accumulators (TMEM lanes
// 32 * (warp % 4); two warps share a quarter and take turns at its column
// blocks), row loads.
constexpr int WARP_A = 0, WARP_MMA = 1, WARP_EPI = 2, EPI_WARPS = 8, WARP_B = WARP_EPI + EPI_WARPS;
constexpr int FFN_WARPS = WARP_B + 1;
constexpr int FFN_THREADS = FFN_WARPS * 32;
constexpr int EPI_THREADS = EPI_WARPS * 32;

constexpr int STEP_BYTES = 32768;  // weights of one step
constexpr int ACC_COLS = 256;      // weight columns of a tile: two accumulators of 128
constexpr int GROUP8 = 128;        // rows and columns of an 8-bit scale block
constexpr int FFN_MAX_STAGES = 6;
constexpr int FFN_MAX_BUFS = 8;
constexpr int RING_BYTES = FFN_MAX_STAGES * (STEP_BYTES + 16 * 128 * 2);  // six stages at up to 16 rows an expert
// 8 bits: the scales of a step (up to 128 rows, then the two weight blocks) in
// a ring of their own at the end, longer than the stages and accumulator
// buffers that lie between their load and their use.
constexpr int SCALE_SLOTS = 16, SCALE_FLOATS = FFN_MAX_T + 4;
constexpr int SCALE_AT = RING_BYTES - SCALE_SLOTS * SCALE_FLOATS * 4;
static_assert(SCALE_SLOTS >= FFN_MAX_STAGES + FFN_MAX_BUFS && SCALE_AT % 16 == 0, "scale ring");
constexpr int MAX_TILES1 = MAX_E * (32768 / 128);
constexpr int SLOTS = 5;           // per CTA: h pieces (first, last range; whole tile), output pieces (first, last)
constexpr long long FFN_SPIN_NS = 2000000000LL;
constexpr float E4M3_TOP = 448.f;
constexpr float TINY = 7.888609052210118e-31f;  // 2^-100

struct FfnCtl {
    uint32_t routed;  // CTAs whose tokens are routed
    uint32_t done;    // CTAs whose output pieces are written
    uint32_t exited;
    uint32_t abort;
    uint32_t pad[60];
    uint32_t ready[MAX_E];            // tiles of h published, per chosen expert
    uint32_t arrived[MAX_TILES1];     // pieces of an h tile delivered
};

struct FfnParams {
    const float* logits;
    const float* x_scale;
    const float* w1_scale;
    const float* w3_scale;
    const float* w2_scale;
    __nv_bfloat16* out;
    FfnCtl* ctl;
    uint8_t* ids;       // [T*k] chosen experts, and
    float* gates;       // [T*k] their gates (when routing is shared out)
    uint8_t* h;         // [2][T*k][F] bf16 (value and remainder) or [T*k][F] e4m3
    float* h_scale;     // [T*k][F/128]
    float* y;           // [T*k][H] products of tiles that one CTA computed whole
    float* slots;       // [ctas][SLOTS][T][256] pieces
    DevError* err;
    int T, H, F, E, k;
};

struct FfnMaps {
    CUtensorMap x, w1, w3, w2, h;
};

struct FfnSmem {
    uint64_t weights_in[FFN_MAX_STAGES], rows_in[FFN_MAX_STAGES], empty[FFN_MAX_STAGES];
    uint64_t acc_full[FFN_MAX_BUFS], acc_empty[FFN_MAX_BUFS];
    uint64_t scales_in[SCALE_SLOTS], scales_out[SCALE_SLOTS];
    uint64_t drain;
    uint32_t tmem_base;
    int ok, last, chosen, most;  // most: rows of the busiest expert
    int scan[8];
    float red[2][2][4];
    uint16_t off[MAX_E + 1];       // per chosen expert: its first row,
    uint8_t expert[MAX_E];         // its id
    uint8_t count[MAX_E];          // and its rows
    uint8_t row_token[FFN_MAX_ROWS];
    uint16_t row_of[FFN_MAX_ROWS]; // per (token, choice): its row,
    uint8_t act_of[FFN_MAX_ROWS];  // its place among the chosen experts
    float gate[FFN_MAX_ROWS];      // and its gate
};
constexpr int FFN_SMEM = RING_BYTES + int(sizeof(FfnSmem)) + 1024;
static_assert(FFN_SMEM <= 232448, "dynamic shared memory of one CTA on sm_103");

// Routing scratch, in the ring before the first load.
constexpr int RS_IDS = 0, RS_MASK = FFN_MAX_ROWS, RS_PLACE = RS_MASK + MAX_E * (FFN_MAX_T / 8);

// One half of the layer as seen by this CTA: steps [start, end) of `total`.
struct Half {
    uint32_t ks;      // steps per tile
    uint32_t blocks;  // tiles per expert
    uint32_t total, ctas, start, end;
    uint32_t each, more;  // steps per CTA; the first `more` CTAs take one more
    __device__ uint32_t first_step(uint32_t c) const { return c * each + min(c, more); }
    __device__ uint32_t owner(uint32_t step) const {
        const uint32_t in_more = more * (each + 1);
        return step < in_more ? step / (each + 1) : more + (step - in_more) / each;
    }
};

__device__ __forceinline__ Half make_half(uint32_t ks, uint32_t blocks, uint32_t experts) {
    Half h;
    h.ks = ks;
    h.blocks = blocks;
    h.total = ks * blocks * experts;
    h.ctas = min(gridDim.x, h.total);  // every CTA that takes part has a step
    h.each = h.total / h.ctas;
    h.more = h.total - h.each * h.ctas;
    const bool in = blockIdx.x < h.ctas;
    h.start = in ? h.first_step(blockIdx.x) : 0u;
    h.end = in ? h.first_step(blockIdx.x + 1) : 0u;
    return h;
}

// Steps [k0, k1) of one tile.
struct Piece {
    uint32_t tile, k0, k1;
    int a, blk;  // place of the expert, block of columns
};

__device__ __forceinline__ bool next_piece(const Half& h, uint32_t& pos, Piece& s) {
    if (pos >= h.end) return false;
    s.tile = pos / h.ks;
    s.k0 = pos - s.tile * h.ks;
    s.k1 = min(h.ks, s.k0 + (h.end - pos));
    s.a = int(s.tile / h.blocks);
    s.blk = int(s.tile - uint32_t(s.a) * h.blocks);
    pos += s.k1 - s.k0;
    return true;
}

__device__ __forceinline__ uint8_t* ffn_ring() {
    extern __shared__ uint8_t ffn_raw[];
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ffn_raw) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ int pad16(int n) { return (n + 15) & ~15; }

template <int ID, int N>
__device__ __forceinline__ void bar_sync() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(N) : "memory");
}

__device__ __forceinline__ float nan_max(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ------------------------------------------------------------- routing -----

// Order of the logits as unsigned integers, above 0: -0 counts as 0, NaN as -inf.
__device__ __forceinline__ uint32_t ordered(float v) {
    if (v != v) v = -INFINITY;
    const uint32_t u = __float_as_uint(v + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

// One token by one warp: the k largest logits in descending order, ties to
// the lower expert, and the softmax over them (0 where the logit is -inf).
__device__ void route_token(const FfnParams& p, int t, uint8_t* ids, float* gates) {
    const int lane = threadIdx.x & 31;
    const float* row = p.logits + size_t(t) * p.E;
    uint32_t key[MAX_E / 32];
#pragma unroll
    for (int i = 0; i < MAX_E / 32; ++i) key[i] = lane + 32 * i < p.E ? ordered(__ldg(row + lane + 32 * i)) : 0u;
    float value = -INFINITY;
    int id = 0;
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < MAX_E / 32; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const int e = int(__reduce_min_sync(0xffffffffu, best == top ? uint32_t(at) : 0xffffu));
#pragma unroll
        for (int i = 0; i < MAX_E / 32; ++i)
            if (lane + 32 * i == e) key[i] = 0;
        if (lane == j) {
            value = unordered(top);
            id = e;
        }
    }
    const float v0 = __shfl_sync(0xffffffffu, value, 0);
    const float w = lane < p.k && value > -INFINITY ? expf(value - v0) : 0.f;
    float sum = 0.f;
    for (int j = 0; j < p.k; ++j) sum += __shfl_sync(0xffffffffu, w, j);
    if (lane < p.k) {
        ids[t * p.k + lane] = uint8_t(id);
        gates[t * p.k + lane] = sum > 0.f ? w / sum : 0.f;
    }
}

// The tables of every CTA from the chosen experts in the scratch: rows sorted
// by (expert, token).  An expert's tokens are a bit mask, so a row's place is
// a count of bits and no order of arrival matters.
__device__ void build_rows(const FfnParams& p, FfnSmem* sm, uint8_t* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int WORDS = FFN_MAX_T / 32;
    const uint8_t* ids = scratch + RS_IDS;
    uint32_t* mask = reinterpret_cast<uint32_t*>(scratch + RS_MASK);
    uint8_t* place = scratch + RS_PLACE;
    const int rows = p.T * p.k;
    for (int i = tid; i < p.E * WORDS; i += FFN_THREADS) mask[i] = 0;
    if (tid == 0) sm->most = 0;
    __syncthreads();
    for (int i = tid; i < rows; i += FFN_THREADS) {
        const int t = i / p.k;
        atomicOr(&mask[ids[i] * WORDS + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    // rows and chosen experts before each expert, 16 bits each
    uint32_t mine = 0;
    if (tid < p.E) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) c += __popc(mask[tid * WORDS + w]);
        mine = uint32_t(c) | (c ? 1u << 16 : 0u);
    }
    uint32_t run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += o;
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, mine & 0xffffu);
    if (warp < MAX_E / 32) {
        if (lane == 31) sm->scan[warp] = int(run);
        if (lane == 0) atomicMax(&sm->most, int(top));
    }
    __syncthreads();
    if (tid < MAX_E) {
        uint32_t base = run - mine;
        for (int w = 0; w < warp; ++w) base += uint32_t(sm->scan[w]);
        const int a = int(base >> 16);
        if (mine) {
            sm->expert[a] = uint8_t(tid);
            sm->count[a] = uint8_t(mine & 0xffffu);
            sm->off[a] = uint16_t(base & 0xffffu);
            place[tid] = uint8_t(a);
        }
        if (tid == MAX_E - 1) sm->chosen = int((base + mine) >> 16);
    }
    __syncthreads();
    for (int i = tid; i < rows; i += FFN_THREADS) {
        const int t = i / p.k, e = ids[i], a = place[e];
        int before = 0;
        for (int w = 0; w < (t >> 5); ++w) before += __popc(mask[e * WORDS + w]);
        before += __popc(mask[e * WORDS + (t >> 5)] & ((1u << (t & 31)) - 1u));
        const int r = sm->off[a] + before;
        sm->row_of[i] = uint16_t(r);
        sm->act_of[i] = uint8_t(a);
        sm->row_token[r] = uint8_t(t);
    }
}

// --------------------------------------------------------------- roles -----

struct Ring {
    uint32_t stages, stage_bytes, bufs, acc_stride;  // acc_stride: TMEM columns of one accumulator
};

struct Turn {  // position in a ring of n slots
    uint32_t i = 0, phase = 0;
    __device__ void next(uint32_t n) {
        if (++i == n) {
            i = 0;
            phase ^= 1u;
        }
    }
};

// The stages that a loading warp has issued, so that after a wait gave up it
// can let its loads land before the CTA exits.
struct Issued {
    uint32_t any = 0, parity = 0;  // per stage: issued at all, the phase of its last load
    __device__ void note(const Turn& t) {
        any |= 1u << t.i;
        parity = (parity & ~(1u << t.i)) | (t.phase << t.i);
    }
    __device__ void settle(uint64_t* bars) const {
        const uint64_t t0 = globaltimer();
        for (uint32_t i = 0; i < FFN_MAX_STAGES; ++i)
            if (any >> i & 1u)
                while (!mbar_try_wait(&bars[i], parity >> i & 1u) && globaltimer() - t0 < 5000000ull) {
                }
        __syncwarp();
    }
};

template <bool FP8>
__device__ void weight_loads(const FfnParams& p, const FfnMaps& m, FfnSmem* sm, const Ring& rg, const Half (&half)[2],
                             const Waiter& w) {
    constexpr int KB = FP8 ? 128 : 64;   // rows of K in a step
    constexpr int CB = FP8 ? 128 : 64;   // columns of a box
    constexpr int BOX = KB * 128;        // bytes of a box
    uint8_t* ring = ffn_ring();
    const uint64_t pol = l2_policy_evict_first();  // every weight is read once
    Turn st;
    Issued mine;
    for (int ph = 0; ph < 2; ++ph) {
        const int ncol = ph == 0 ? p.F : p.H, krows = ph == 0 ? p.H : p.F;
        uint32_t pos = half[ph].start;
        Piece s;
        while (next_piece(half[ph], pos, s)) {
            const int row0 = sm->expert[s.a] * krows;
            for (uint32_t k = s.k0; k < s.k1; ++k) {
                if (!warp_await_mbar(&sm->empty[st.i], st.phase ^ 1u, w, SITE_STAGE_EMPTY)) {
                    mine.settle(sm->weights_in);
                    return;
                }
                uint64_t* fb = &sm->weights_in[st.i];
                uint8_t* dst = ring + st.i * rg.stage_bytes;
                mine.note(st);
                mbar_arrive_expect_tx_elect(fb, STEP_BYTES);
                const int row = row0 + int(k) * KB;
#pragma unroll
                for (int q = 0; q < STEP_BYTES / BOX; ++q) {
                    // boxes past the matrix's edge read as zeros
                    const int c = ph == 0 ? s.blk * 128 + (q * CB) % 128 : s.blk * ACC_COLS + q * CB;
                    const CUtensorMap* map = ph == 1 ? &m.w2 : q * CB < 128 ? &m.w1 : &m.w3;
                    tma_load_2d_elect_hint(dst + q * BOX, map, c < ncol ? c : ncol, row, fb, pol);
                }
                st.next(rg.stages);
            }
        }
    }
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <bool FP8>
__device__ void row_loads(const FfnParams& p, const FfnMaps& m, FfnSmem* sm, const Ring& rg, const Half (&half)[2],
                          const Waiter& w) {
    constexpr int KB = FP8 ? 128 : 64;
    const int lane = threadIdx.x & 31;
    uint8_t* ring = ffn_ring();
    Turn st, sc;
    Issued mine;
    auto leave = [&]() {
        if (FP8) cp_async_wait_all();
        mine.settle(sm->rows_in);
    };
    for (int ph = 0; ph < 2; ++ph) {
        uint32_t pos = half[ph].start;
        Piece s;
        int known = -1;
        const int parts = ph == 1 && !FP8 ? 2 : 1;  // h: value and remainder
        while (next_piece(half[ph], pos, s)) {
            const int n = sm->count[s.a], N = pad16(n), off = sm->off[s.a];
            if (ph == 1 && s.a != known) {
                const bool in = await_geq(&p.ctl->ready[s.a], half[0].blocks, w, SITE_TILE_READY);
                if (!__all_sync(0xffffffffu, in)) {
                    leave();
                    return;
                }
                fence_proxy_async();  // the other CTAs' stores to h before the loads below
                known = s.a;
            }
            int r[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = off + min(4 * lane + q, n - 1);  // rows past the last repeat it; never stored
                r[q] = ph == 0 ? sm->row_token[i] : i;
            }
            // 8 bits: scales of this lane's rows lane, lane + 32, ... and of the two weight blocks
            const int KB8 = (ph == 0 ? p.H : p.F) / GROUP8, NB8 = (ph == 0 ? p.F : p.H) / GROUP8;
            const float* sx[FFN_MAX_T / 32];
            const float* sw = nullptr;
            if constexpr (FP8) {
#pragma unroll
                for (int q = 0; q < FFN_MAX_T / 32; ++q) {
                    const int i = off + min(lane + 32 * q, n - 1);
                    sx[q] = ph == 0 ? p.x_scale + size_t(sm->row_token[i]) * KB8 : p.h_scale + size_t(i) * KB8;
                }
                const size_t block = size_t(sm->expert[s.a]) * KB8 * NB8;
                if (ph == 0) sw = (lane == 0 ? p.w1_scale : p.w3_scale) + block + s.blk;
                else sw = p.w2_scale + block + min(2 * s.blk + (lane & 1), NB8 - 1);
            }
            for (uint32_t k = s.k0; k < s.k1; ++k) {
                if (!warp_await_mbar(&sm->empty[st.i], st.phase ^ 1u, w, SITE_STAGE_EMPTY)) {
                    leave();
                    return;
                }
                uint64_t* fb = &sm->rows_in[st.i];
                uint8_t* dst = ring + st.i * rg.stage_bytes + STEP_BYTES;
                mine.note(st);
                mbar_arrive_expect_tx_elect(fb, uint32_t(N * 128 * parts));
                __syncwarp();
                if (4 * lane < N) {
                    tma_gather4(dst + lane * 512, ph == 0 ? &m.x : &m.h, int(k) * KB, r[0], r[1], r[2], r[3], fb);
                    if (parts == 2) {
                        const int R = p.T * p.k;
                        tma_gather4(dst + N * 128 + lane * 512, &m.h, int(k) * KB, R + r[0], R + r[1], R + r[2],
                                    R + r[3], fb);
                    }
                }
                if constexpr (FP8) {
                    if (!warp_await_mbar(&sm->scales_out[sc.i], sc.phase ^ 1u, w, SITE_ACC_EMPTY)) {
                        leave();
                        return;
                    }
                    const uint32_t to = smem_u32(ring + SCALE_AT) + sc.i * (SCALE_FLOATS * 4);
#pragma unroll
                    for (int q = 0; q < FFN_MAX_T / 32; ++q)
                        if (lane + 32 * q < N) cp_async_4(to + (lane + 32 * q) * 4, sx[q] + k);
                    if (lane < 2) cp_async_4(to + (FFN_MAX_T + lane) * 4, sw + size_t(k) * NB8);
                    cp_async_mbar_arrive_noinc(&sm->scales_in[sc.i]);
                    sc.next(SCALE_SLOTS);
                }
                __syncwarp();
                st.next(rg.stages);
            }
        }
    }
}

template <bool FP8>
__device__ void products(FfnSmem* sm, const Ring& rg, const Half (&half)[2], const Waiter& w) {
    const uint32_t ring = smem_u32(ffn_ring());
    Turn st, buf;
    bool issued = false, ok = true;
    for (int ph = 0; ph < 2 && ok; ++ph) {
        uint32_t pos = half[ph].start;
        Piece s;
        while (ok && next_piece(half[ph], pos, s)) {
            const uint32_t N = uint32_t(pad16(sm->count[s.a]));
            const uint32_t idesc = FP8 ? umma_idesc_e4m3(128, N, true, false) : umma_idesc_bf16(128, N, true, false);
            for (uint32_t k = s.k0; k < s.k1; ++k) {
                // 16 bits: one accumulation per piece; 8 bits: one per step
                if (FP8 || k == s.k0) {
                    if (!(ok = warp_await_mbar(&sm->acc_empty[buf.i], buf.phase ^ 1u, w, SITE_ACC_EMPTY))) break;
                }
                if (!(ok = warp_await_mbar(&sm->rows_in[st.i], st.phase, w, SITE_STAGE_FULL))) break;
                if (!(ok = warp_await_mbar(&sm->weights_in[st.i], st.phase, w, SITE_STAGE_FULL))) break;
                tc_fence_after();
                const uint32_t d = sm->tmem_base + buf.i * 2u * rg.acc_stride;
                const uint32_t a = ring + st.i * rg.stage_bytes, b = a + STEP_BYTES;
                issued = true;
                if constexpr (FP8) {
                    // 128 columns of weights are one swizzle span; K rows in groups of 8,
                    // 1024 bytes apart: 4 KiB per K = 32
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t bd = umma_desc_sw128(b + kk * 32, 16, 1024);
                        tc_mma_f8_elect(d, umma_desc_sw128(a + kk * 4096, 16384, 1024), bd, idesc, kk != 0);
                        tc_mma_f8_elect(d + rg.acc_stride, umma_desc_sw128(a + 16384 + kk * 4096, 16384, 1024), bd,
                                        idesc, kk != 0);
                    }
                } else {
                    // two 64-column chunks 8 KiB apart; 2 KiB per K = 16
                    const int parts = ph + 1;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t a0 = umma_desc_sw128(a + kk * 2048, 8192, 1024);
                        const uint64_t a1 = umma_desc_sw128(a + 16384 + kk * 2048, 8192, 1024);
                        for (int q = 0; q < parts; ++q) {
                            const uint64_t bd = umma_desc_sw128(b + q * N * 128 + kk * 32, 16, 1024);
                            const uint32_t add = k != s.k0 || kk != 0 || q != 0;
                            tc_mma_f16_elect(d, a0, bd, idesc, add);
                            tc_mma_f16_elect(d + rg.acc_stride, a1, bd, idesc, add);
                        }
                    }
                }
                tc_commit_elect(&sm->empty[st.i]);
                st.next(rg.stages);
                if (FP8 || k + 1 == s.k1) {
                    tc_commit_elect(&sm->acc_full[buf.i]);
                    buf.next(rg.bufs);
                }
            }
        }
    }
    if (issued) {
        // every product has completed before TMEM is freed
        tc_commit_elect(&sm->drain);
        const uint64_t t0 = globaltimer();
        while (!__all_sync(0xffffffffu, mbar_try_wait(&sm->drain, 0u)) && globaltimer() - t0 < 5000000ull) {
        }
    }
    __syncwarp();
}

__device__ __forceinline__ float* slot_of(const FfnParams& p, uint32_t cta, int which) {
    return p.slots + (size_t(cta) * SLOTS + which) * size_t(p.T) * ACC_COLS;
}

// Pieces of a tile: CTAs [c0, c0 + n); the piece of CTA c lies in its slot
// `first` if the tile holds the CTA's first step, else in the next one.
struct Pieces {
    uint32_t c0, n, begin;
};
__device__ __forceinline__ Pieces pieces_of(const Half& h, uint32_t tile) {
    Pieces q;
    q.begin = tile * h.ks;
    q.c0 = h.owner(q.begin);
    q.n = h.owner(q.begin + h.ks - 1) - q.c0 + 1;
    return q;
}
__device__ __forceinline__ const float* piece(const FfnParams& p, const Half& h, const Pieces& q, uint32_t i,
                                              int first) {
    const uint32_t c = q.c0 + i;
    return slot_of(p, c, first + (h.first_step(c) >= q.begin ? 0 : 1));
}

// h of a complete tile from its pieces, by the eight draining warps.
template <bool FP8>
__device__ void finish_tile(const FfnParams& p, FfnSmem* sm, const Half& hf, const Piece& s, const Pieces& q) {
    const int et = threadIdx.x - WARP_EPI * 32, f = et & 127, side = et >> 7;
    const int n = sm->count[s.a], off = sm->off[s.a], col = s.blk * 128 + f;
    const size_t R = size_t(p.T) * p.k;
    for (int i = side; i < n; i += 2) {
        float a = 0.f, b = 0.f;
        for (uint32_t j = 0; j < q.n; ++j) {
            const float* src = q.n == 1 ? slot_of(p, q.c0, 2) : piece(p, hf, q, j, 0);
            a += __ldcg(src + size_t(i) * ACC_COLS + f);
            b += __ldcg(src + size_t(i) * ACC_COLS + 128 + f);
        }
        const float v = a / (1.f + expf(-a)) * b;
        const size_t at = size_t(off + i) * p.F + col;
        if constexpr (FP8) {
            float top = fabsf(v);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = nan_max(top, __shfl_xor_sync(0xffffffffu, top, d));
            float* red = sm->red[side][(i >> 1) & 1];
            if ((f & 31) == 0) red[f >> 5] = top;
            if (side == 0) bar_sync<2, 128>();
            else bar_sync<3, 128>();
            top = nan_max(nan_max(red[0], red[1]), nan_max(red[2], red[3]));
            const float scale = top < TINY ? 1.f : top / E4M3_TOP;
            p.h[at] = uint8_t(__nv_cvt_float_to_fp8(v * (1.f / scale), __NV_SATFINITE, __NV_E4M3));
            if (f == 0) p.h_scale[size_t(off + i) * (p.F / GROUP8) + s.blk] = scale;
        } else if (col < p.F) {
            const __nv_bfloat16 hi = __float2bfloat16_rn(v);
            __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(p.h);
            h[at] = hi;
            h[R * p.F + at] = __float2bfloat16_rn(v - __bfloat162float(hi));
        }
    }
}

template <bool FP8>
__device__ void drain_accumulators(const FfnParams& p, FfnSmem* sm, const Ring& rg, const Half (&half)[2],
                                   const Waiter& w) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, set = (warp - WARP_EPI) >> 2;
    const int et = threadIdx.x - WARP_EPI * 32;
    constexpr int MAXB = FFN_MAX_T / 32;  // blocks of 16 columns per warp
    const uint32_t tq = sm->tmem_base + (uint32_t(quad * 32) << 16);
    Turn buf, sc;
    // A wait that gave up only stops the work: the barriers that the eight
    // warps share are still reached by all of them.
    bool ok = true;
    for (int ph = 0; ph < 2; ++ph) {
        const Half& hf = half[ph];
        uint32_t pos = hf.start;
        Piece s;
        while (next_piece(hf, pos, s)) {
            const int n = sm->count[s.a], off = sm->off[s.a];
            const int nblk = pad16(n) / 16;
            const Pieces q = pieces_of(hf, s.tile);
            const bool whole = q.n == 1;
            // where the sums go: row i, this lane's columns f (first accumulator) and 128 + f
            const int f = quad * 32 + lane;
            float* dst;
            size_t stride = ACC_COLS;
            bool in0 = true, in1 = true;
            if (ph == 1 && whole) {
                const int col = s.blk * ACC_COLS + f;
                dst = p.y + size_t(off) * p.H + col;
                stride = size_t(p.H);
                in0 = col < p.H;
                in1 = col + 128 < p.H;
            } else {
                const int which = ph == 0 ? (whole ? 2 : hf.start >= q.begin ? 0 : 1) : (hf.start >= q.begin ? 3 : 4);
                dst = slot_of(p, blockIdx.x, which) + f;
            }
            auto put = [&](int blk, const float (&v0)[16], const float (&v1)[16]) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = blk * 16 + i;
                    if (r < n) {
                        float* d = dst + size_t(r) * stride;
                        if (in0) __stcg(d, v0[i]);
                        if (in1) __stcg(d + 128, v1[i]);
                    }
                }
            };
            if constexpr (!FP8) {
                if (ok) ok = warp_await_mbar(&sm->acc_full[buf.i], buf.phase, w, SITE_ACC_FULL);
                if (ok) {
                    tc_fence_after();
                    const uint32_t t0 = tq + buf.i * 2u * rg.acc_stride;
                    for (int blk = set; blk < nblk; blk += 2) {
                        uint32_t r0[16], r1[16];
                        tmem_ld_32x32b_x16(t0 + blk * 16, r0);
                        tmem_ld_32x32b_x16(t0 + rg.acc_stride + blk * 16, r1);
                        tmem_ld_wait();
                        float v0[16], v1[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            v0[i] = __uint_as_float(r0[i]);
                            v1[i] = __uint_as_float(r1[i]);
                        }
                        put(blk, v0, v1);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm->acc_empty[buf.i]);
                }
                buf.next(rg.bufs);
            } else {
                float acc0[MAXB][16], acc1[MAXB][16];
#pragma unroll
                for (int b = 0; b < MAXB; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc0[b][i] = acc1[b][i] = 0.f;
                for (uint32_t k = s.k0; k < s.k1; ++k) {
                    if (ok) ok = warp_await_mbar(&sm->scales_in[sc.i], sc.phase, w, SITE_ACC_FULL);
                    if (ok) ok = warp_await_mbar(&sm->acc_full[buf.i], buf.phase, w, SITE_ACC_FULL);
                    if (ok) {
                        tc_fence_after();
                        const uint32_t t0 = tq + buf.i * 2u * rg.acc_stride;
                        const float* scale =
                            reinterpret_cast<const float*>(ffn_ring() + SCALE_AT) + sc.i * SCALE_FLOATS;
                        const float c0 = scale[FFN_MAX_T], c1 = scale[FFN_MAX_T + 1];
#pragma unroll
                        for (int b = 0; b < MAXB; ++b) {
                            const int blk = set + 2 * b;
                            if (blk < nblk) {
                                uint32_t r0[16], r1[16];
                                tmem_ld_32x32b_x16(t0 + blk * 16, r0);
                                tmem_ld_32x32b_x16(t0 + rg.acc_stride + blk * 16, r1);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float x = scale[blk * 16 + i];
                                    acc0[b][i] = fmaf(__uint_as_float(r0[i]), x * c0, acc0[b][i]);
                                    acc1[b][i] = fmaf(__uint_as_float(r1[i]), x * c1, acc1[b][i]);
                                }
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sm->acc_empty[buf.i]);
                            mbar_arrive(&sm->scales_out[sc.i]);
                        }
                    }
                    buf.next(rg.bufs);
                    sc.next(SCALE_SLOTS);
                }
                if (ok) {
#pragma unroll
                    for (int b = 0; b < MAXB; ++b)
                        if (set + 2 * b < nblk) put(set + 2 * b, acc0[b], acc1[b]);
                }
            }
            if (ph == 0) {
                // the CTA that delivers a tile's last piece completes the tile
                __threadfence();
                bar_sync<1, EPI_THREADS>();
                if (!whole) {
                    if (et == 0) {
                        uint32_t* a = &p.ctl->arrived[s.tile];
                        const bool last = atom_add_acq_rel_u32(a, 1u) == q.n - 1;
                        if (last) *a = 0u;
                        sm->last = last;
                        __threadfence();
                    }
                    bar_sync<1, EPI_THREADS>();
                }
                if (whole || sm->last) {
                    finish_tile<FP8>(p, sm, hf, s, q);
                    __threadfence();
                    fence_proxy_async();
                    bar_sync<1, EPI_THREADS>();
                    if (et == 0 && ok) atom_add_acq_rel_u32(&p.ctl->ready[s.a], 1u);
                }
            }
        }
    }
    __threadfence();
}

// out[t] = sum over the k choices, in order, of gate * (the row's pieces, in order).
__device__ void combine_rows(const FfnParams& p, const FfnSmem* sm, const Half& hf) {
    const int lane = threadIdx.x & 31;
    const int nb = (p.H + 127) / 128;
    for (int item = blockIdx.x * FFN_WARPS + (threadIdx.x >> 5); item < p.T * nb; item += gridDim.x * FFN_WARPS) {
        const int t = item / nb, cb = item - t * nb, col = cb * 128 + lane * 4;
        if (col >= p.H) continue;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < p.k; ++j) {
            const int i = t * p.k + j, a = sm->act_of[i], r = sm->row_of[i];
            const Pieces q = pieces_of(hf, uint32_t(a) * hf.blocks + uint32_t(cb >> 1));
            float4 v;
            if (q.n == 1) {
                v = __ldcg(reinterpret_cast<const float4*>(p.y + size_t(r) * p.H + col));
            } else {
                v = make_float4(0.f, 0.f, 0.f, 0.f);
                const size_t at = size_t(r - sm->off[a]) * ACC_COLS + (cb & 1) * 128 + lane * 4;
                for (uint32_t c = 0; c < q.n; ++c) {
                    const float4 u = __ldcg(reinterpret_cast<const float4*>(piece(p, hf, q, c, 3) + at));
                    v.x += u.x;
                    v.y += u.y;
                    v.z += u.z;
                    v.w += u.w;
                }
            }
            const float g = sm->gate[i];
            acc.x = fmaf(g, v.x, acc.x);
            acc.y = fmaf(g, v.y, acc.y);
            acc.z = fmaf(g, v.z, acc.z);
            acc.w = fmaf(g, v.w, acc.w);
        }
        const __nv_bfloat162 b0 = __floats2bfloat162_rn(acc.x, acc.y), b1 = __floats2bfloat162_rn(acc.z, acc.w);
        *reinterpret_cast<uint2*>(p.out + size_t(t) * p.H + col) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
    }
}

template <bool FP8>
__global__ void __launch_bounds__(FFN_THREADS, 1)
    mk_moe_ffn_decode_kernel(const FfnParams p, const __grid_constant__ FfnMaps m) {
    uint8_t* ring = ffn_ring();
    FfnSmem* sm = reinterpret_cast<FfnSmem*>(ring + RING_BYTES);
    const int tid = threadIdx.x, warp = tid >> 5;
    const Waiter w{p.err, &p.ctl->abort, FFN_SPIN_NS};
    // waits inside the pipeline stall because something upstream does: they
    // get longer, so that the one that is recorded is the one at the root
    const Waiter wp{p.err, &p.ctl->abort, 2 * FFN_SPIN_NS};

    if (tid == 0) {
        for (int i = 0; i < FFN_MAX_STAGES; ++i) {
            mbar_init(&sm->weights_in[i], 1);
            mbar_init(&sm->rows_in[i], 1);
            mbar_init(&sm->empty[i], 1);
        }
        for (int i = 0; i < FFN_MAX_BUFS; ++i) {
            mbar_init(&sm->acc_full[i], 1);
            mbar_init(&sm->acc_empty[i], EPI_WARPS);
        }
        for (int i = 0; i < SCALE_SLOTS; ++i) {
            mbar_init(&sm->scales_in[i], 32);
            mbar_init(&sm->scales_out[i], EPI_WARPS);
        }
        mbar_init(&sm->drain, 1);
        fence_barrier_init();
        sm->ok = 1;
        tma_prefetch_desc(&m.w1);
        tma_prefetch_desc(&m.w3);
        tma_prefetch_desc(&m.x);
    }
    if (warp == WARP_MMA) {
        tmem_alloc(&sm->tmem_base, 512);
        tmem_relinquish();
    }

    // ---- routing: a warp per token, in every CTA for itself, or shared out
    // over the CTAs and read back after a barrier once there are more tokens
    // than a CTA has warps (a second token per warp would cost about what the
    // barrier does)
    uint8_t* ids = ring + RS_IDS;
    const int rows = p.T * p.k;
    if (p.T <= FFN_WARPS) {
        if (warp < p.T) route_token(p, warp, ids, sm->gate);
        __syncthreads();
    } else {
        for (int t = blockIdx.x + int(gridDim.x) * warp; t < p.T; t += int(gridDim.x) * FFN_WARPS)
            route_token(p, t, p.ids, p.gates);
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            atom_add_acq_rel_u32(&p.ctl->routed, 1u);
            sm->ok = await_geq(&p.ctl->routed, gridDim.x, w, SITE_BAR_ROUTED);
        }
        __syncthreads();
        for (int i = tid; i < rows; i += FFN_THREADS) {
            ids[i] = __ldcg(p.ids + i);
            sm->gate[i] = __ldcg(p.gates + i);
        }
        __syncthreads();
    }
    if (sm->ok) {
        build_rows(p, sm, ring);
        fence_proxy_async_shared();  // the scratch's generic accesses before TMA writes there
        tc_fence_before();
        __syncthreads();
        tc_fence_after();

        constexpr int KB = FP8 ? 128 : 64;
        const Half half[2] = {make_half(p.H / KB, (p.F + 127) / 128, sm->chosen),
                              make_half(p.F / KB, (p.H + ACC_COLS - 1) / ACC_COLS, sm->chosen)};
        Ring rg;
        const int N = pad16(sm->most);
        rg.acc_stride = uint32_t(N);
        rg.stage_bytes = uint32_t(STEP_BYTES + N * 128 * (FP8 ? 1 : 2));
        rg.stages = min(uint32_t(FFN_MAX_STAGES), uint32_t(FP8 ? SCALE_AT : RING_BYTES) / rg.stage_bytes);
        rg.bufs = FP8 ? min(uint32_t(FFN_MAX_BUFS), 512u / (2u * rg.acc_stride)) : 2u;

        if (warp == WARP_A) weight_loads<FP8>(p, m, sm, rg, half, wp);
        else if (warp == WARP_B) row_loads<FP8>(p, m, sm, rg, half, w);
        else if (warp == WARP_MMA) products<FP8>(sm, rg, half, wp);
        else drain_accumulators<FP8>(p, sm, rg, half, wp);

        __syncthreads();
        if (tid == 0) {
            __threadfence();
            atom_add_acq_rel_u32(&p.ctl->done, 1u);
            sm->ok = await_geq(&p.ctl->done, gridDim.x, w, SITE_BAR_COMPUTED) && ld_relaxed_u32(w.abort) == 0u;
        }
        __syncthreads();
        if (sm->ok) combine_rows(p, sm, half[1]);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc(sm->tmem_base, 512);
    }
    if (tid == 0 && atom_add_acq_rel_u32(&p.ctl->exited, 1u) == gridDim.x - 1) {
        // the last CTA out leaves the control block ready for the next call
        FfnCtl* c = p.ctl;
        c->routed = 0;
        c->done = 0;
        for (int i = 0; i < MAX_E; ++i) c->ready[i] = 0;
        if (c->abort != 0)
            for (int i = 0; i < MAX_TILES1; ++i) c->arrived[i] = 0;  // a call that gave up left some
        c->abort = 0;
        c->exited = 0;
        __threadfence();
    }
}

struct FfnLayout {
    size_t ctl, ids, gates, h, h_scale, y, slots, total;
};

FfnLayout ffn_layout(int T, int H, int F, int k, bool fp8) {
    const size_t R = size_t(T) * k;
    FfnLayout L{};
    size_t o = 0;
    L.ctl = o;      o = ws_align(o + sizeof(FfnCtl));
    L.ids = o;      o = ws_align(o + R);
    L.gates = o;    o = ws_align(o + R * 4);
    L.h = o;        o = ws_align(o + R * F * (fp8 ? 1 : 4));
    L.h_scale = o;  o = ws_align(o + (fp8 ? R * (F / GROUP8) * 4 : 0));
    L.y = o;        o = ws_align(o + R * H * 4);
    L.slots = o;    o = ws_align(o + size_t(FFN_MAX_CTAS) * SLOTS * T * ACC_COLS * 4);
    L.total = o;
    return L;
}

mk_status_t ffn_sizes(int T, int H, int E, int k, int F, int weights) {
    if (T < 0 || E < 1 || k < 1 || k > E || k > MAX_K) return MK_ERR_INVALID_ARG;
    if (weights != MK_WEIGHT_BF16 && weights != MK_WEIGHT_E4M3) return MK_ERR_INVALID_ARG;
    if (E > MAX_E || T > FFN_MAX_T) return MK_ERR_UNSUPPORTED;
    const int unit = weights == MK_WEIGHT_E4M3 ? GROUP8 : 64;
    if (H < unit || F < unit || H % unit != 0 || F % unit != 0) return MK_ERR_INVALID_ARG;
    if (H > 32768 || F > 32768) return MK_ERR_UNSUPPORTED;
    return MK_OK;
}

template <bool FP8>
cudaError_t launch_ffn(const FfnParams& p, const FfnMaps& m, int grid, cudaStream_t st) {
    // the CTAs wait for one another: a cooperative launch has all of them resident
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(FFN_THREADS);
    cfg.dynamicSmemBytes = FFN_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mk_moe_ffn_decode_kernel<FP8>, p, m);
}

}  // namespace

cudaError_t ffn_kernel_attributes() {
    const cudaError_t e =
        cudaFuncSetAttribute(mk_moe_ffn_decode_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, FFN_SMEM);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(mk_moe_ffn_decode_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, FFN_SMEM);
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_moe_ffn_decode_workspace_size(int T, int H, int F, int E, int k, int weights) {
    if (ffn_sizes(T, H, E, k, F, weights) != MK_OK) return 0;
    return ffn_layout(T, H, F, k, weights == MK_WEIGHT_E4M3).total;
}

extern "C" mk_status_t mk_moe_ffn_decode(const void* x, const float* x_scale, const float* logits, int T, int H, int E,
                                         int k, const void* W1, const void* W3, const void* W2, const float* W1_scale,
                                         const float* W3_scale, const float* W2_scale, int F, int weights, void* out,
                                         void* stream, void* workspace, size_t ws_bytes) {
    mk_status_t s = ffn_sizes(T, H, E, k, F, weights);
    if (s != MK_OK) return s;
    const bool fp8 = weights == MK_WEIGHT_E4M3;
    if (T > 0) {
        if (!x || !logits || !W1 || !W3 || !W2 || !out) return MK_ERR_INVALID_ARG;
        if (!host_aligned(x, 16) || !host_aligned(W1, 16) || !host_aligned(W3, 16) || !host_aligned(W2, 16) ||
            !host_aligned(out, 16) || !host_aligned(logits, 4))
            return MK_ERR_INVALID_ARG;
        const float* scales[4] = {x_scale, W1_scale, W3_scale, W2_scale};
        for (const float* v : scales)
            if ((v != nullptr) != fp8 || !host_aligned(v, 4)) return MK_ERR_INVALID_ARG;
    }
    int dev = 0, sms = 0;
    DevError* err = nullptr;
    if ((s = host_device(&dev, &sms, &err)) != MK_OK) return s;
    if (T == 0) return MK_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const FfnLayout L = ffn_layout(T, H, F, k, fp8);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    if (ws) {
        if (ws_bytes < L.total || !host_aligned(ws, 256)) return MK_ERR_WORKSPACE;
    } else {
        void* v = nullptr;
        if ((s = host_workspace(WS_FFN, dev, st, L.total, L.total, &v)) != MK_OK) return s;
        ws = static_cast<uint8_t*>(v);
    }
    FfnParams p{};
    p.logits = logits;
    p.x_scale = x_scale;
    p.w1_scale = W1_scale;
    p.w3_scale = W3_scale;
    p.w2_scale = W2_scale;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.ctl = reinterpret_cast<FfnCtl*>(ws + L.ctl);
    p.ids = ws + L.ids;
    p.gates = reinterpret_cast<float*>(ws + L.gates);
    p.h = ws + L.h;
    p.h_scale = reinterpret_cast<float*>(ws + L.h_scale);
    p.y = reinterpret_cast<float*>(ws + L.y);
    p.slots = reinterpret_cast<float*>(ws + L.slots);
    p.err = err;
    p.T = T;
    p.H = H;
    p.F = F;
    p.E = E;
    p.k = k;

    const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t size = fp8 ? 1 : 2;
    const uint32_t box = fp8 ? 128 : 64;  // one 128-byte swizzle span, and the rows of K of a step
    const uint64_t R = uint64_t(T) * k * (fp8 ? 1 : 2);
    FfnMaps m;
    std::memset(&m, 0, sizeof(m));
    if (host_encode_2d(&m.x, type, x, H, T, H * size, box, 1) != CUDA_SUCCESS ||
        host_encode_2d(&m.w1, type, W1, F, uint64_t(E) * H, F * size, box, box) != CUDA_SUCCESS ||
        host_encode_2d(&m.w3, type, W3, F, uint64_t(E) * H, F * size, box, box) != CUDA_SUCCESS ||
        host_encode_2d(&m.w2, type, W2, H, uint64_t(E) * F, H * size, box, box) != CUDA_SUCCESS ||
        host_encode_2d(&m.h, type, p.h, F, R, F * size, box, 1) != CUDA_SUCCESS)
        return MK_ERR_CUDA;
    const int grid = std::min(sms, FFN_MAX_CTAS);
    const cudaError_t e = fp8 ? launch_ffn<true>(p, m, grid, st) : launch_ffn<false>(p, m, grid, st);
    return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
